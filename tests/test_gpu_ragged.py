"""The ragged-batch operators on the GPU against their definitions
(oracle/ragged.py): the page plan, append to and read-back from the 8-bit
cache, the attention over it, and the adjustment of logits."""
import numpy as np
import pytest
import torch

import activation_kv_sparsity_b200 as bc
from oracle import ragged as og
from ragged_util import attention_tol, gen, make_pool, to

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------ the plan
def run_plan(lens, delta, table, free_list, n_free, max_tokens, in_place=False):
    d = dict(lens=ints(lens), delta=ints(delta), table=ints(table), free_list=ints(free_list), n_free=ints([n_free]))
    B = len(lens)
    d["lens_out"] = d["lens"] if in_place else ints([-7] * B)
    d["n_free_out"] = d["n_free"] if in_place else ints([-7])
    d["q_start"] = ints([-7] * (B + 1))
    d["slots"], d["positions"] = ints([-7] * max_tokens), ints([-7] * max_tokens)
    d["ticket"] = ints([0])
    bc.block_tables(**d)
    torch.cuda.synchronize()
    assert int(d["ticket"]) == 0
    return dict(table=d["table"], free_list=d["free_list"], n_free=int(d["n_free_out"]), lens=d["lens_out"],
                q_start=d["q_start"], slots=d["slots"], positions=d["positions"])


def check_plan(lens, delta, table, free_list, n_free, max_tokens, in_place=False):
    lens, delta = np.asarray(lens, np.int32), np.asarray(delta, np.int32)
    want = og.block_tables(lens, delta, table, free_list, n_free, max_tokens)
    got = run_plan(lens, delta, table, free_list, n_free, max_tokens, in_place)
    for k, w in want.items():
        g = got[k].cpu().numpy() if isinstance(got[k], torch.Tensor) else got[k]
        np.testing.assert_array_equal(g, w, err_msg=k)
    return want


def fresh(B, max_blocks, n_pages, lens, seed=0):
    rng = np.random.default_rng(seed)
    perm = rng.permutation(n_pages).astype(np.int32)
    table = np.full((B, max_blocks), -1, np.int32)
    at = 0
    for b, n in enumerate(lens):
        p = og.pages_of(n)
        table[b, :p] = perm[at:at + p]
        at += p
    free = np.full(n_pages, -1, np.int32)
    free[:n_pages - at] = perm[at:]
    return table, free, n_pages - at


@pytest.mark.parametrize("B", [1, 2, 7, 33, 1024, 1025, 2048])
@pytest.mark.parametrize("in_place", [False, True])
def test_plan_random_steps(B, in_place):
    rng = np.random.default_rng(B)
    max_blocks = 9
    lens = rng.integers(0, 8 * 16, B)
    table, free, n_free = fresh(B, max_blocks, 9 * B + 3, lens)
    for step in range(4):
        delta = rng.choice([1, 1, 0, 16, 17, 33, -1, -16, -500, 200], B)
        w = check_plan(lens, delta, table, free, n_free, int(max(1, delta[delta > 0].sum() * (0.7 if step == 2 else 1.0))),
                       in_place)
        lens, table, free, n_free = w["lens"], w["table"], w["free_list"], w["n_free"]


@pytest.mark.parametrize("n_free", [0, 1, 2, 5])
def test_plan_refuses_when_pages_run_out(n_free):
    lens = [16, 5, 32, 0, 31, 0]
    table, free, _ = fresh(6, 4, 16, lens)
    w = check_plan(lens, [1, 1, 1, 3, 1, 20], table, free, n_free, 100)
    # the second and the fifth need no page and are never refused
    assert w["q_start"][2] - w["q_start"][1] == 1 and w["q_start"][5] - w["q_start"][4] == 1


def test_plan_gives_back_and_takes_in_one_step():
    lens = [40, 16, 0, 64]
    table, free, n_free = fresh(4, 6, 8, lens)
    assert n_free == 0
    w = check_plan(lens, [-25, 1, 33, -2 ** 31], table, free, n_free, 40)
    assert w["lens"].tolist() == [15, 17, 33, 0]
    check_plan(lens, [-25, 0, 0, -64], table, free, n_free, 40)


def test_plan_limits_of_table_and_tokens():
    table, free, n_free = fresh(3, 2, 12, [0, 30, 4])
    w = check_plan([0, 30, 4], [33, 3, 28], table, free, n_free, 28)       # two over the table
    assert w["q_start"].tolist() == [0, 0, 0, 28]
    w = check_plan([0, 30, 4], [2, 2, 2], table, free, n_free, 4)          # the third over max_tokens
    assert w["q_start"].tolist() == [0, 2, 4, 4]
    check_plan([0, 30, 4], [2, 2, -2], table, free, n_free, 0)
    check_plan([-5, 99, 4], [1, -1, 1], table, free, 10 ** 6, 9)           # lengths and counts out of range


def test_plan_long_prompts():
    lens = [0, 100, 0]
    table, free, n_free = fresh(3, 4000, 9000, lens)
    check_plan(lens, [50001, 1, 60000], table, free, n_free, 111111)


# ------------------------------------------------------------------ the cache
CODES = ["e4m3", "int8"]
DTYPES = [torch.float32, torch.bfloat16]


def blocks_equal(got, want, hd):
    """Codes and scales bit for bit (the padding is not the operator's)."""
    n = 2 * 16 * hd + 8
    np.testing.assert_array_equal(got[..., :n], want[..., :n])


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hd,H", [(64, 2), (128, 3)])
def test_append_codes_exact(code, dtype, hd, H):
    g = gen(hd + H)
    n_pages = 9
    pool = make_pool(n_pages, H, hd, code, seed=5)
    dev = to(DEV, pool)
    # runs: a fresh page filled past its middle, one token into a used page, a run over a page's end,
    # skipped tokens, the last slot of the pool; magnitudes that grow and shrink
    for call, slots in enumerate([[3 * 16 + i for i in range(11)], [3 * 16 + 11], [5 * 16 + 4, 5 * 16 + 5, -1, 10 ** 6, 2 * 16 + 15],
                                  list(range(7 * 16 + 9, 8 * 16 + 7)), [16 * 16], [9 * 16 - 1], [48 + 12, 48 + 13]]):
        n = len(slots)
        amp = [1.0, 50.0, 0.01, 3.0, 1.0, 1e-30, 1e4][call]
        k = (torch.randn(n, H, hd, generator=g) * amp).to(dtype)
        v = (torch.randn(n, H, hd, generator=g) * amp).to(dtype)
        v[0, 0] = 0.0
        og.append(pool, k.float().numpy(), v.float().numpy(), slots, code)
        bc.kv8_append(k.to(DEV), v.to(DEV), ints(slots), dev, code)
        torch.cuda.synchronize()
        blocks_equal(dev.cpu().numpy(), pool, hd)
    assert (dev.cpu().numpy()[..., 2 * 16 * hd + 8:] == 0xA5).all()


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("n", [1, 15, 16, 17, 300, 2048, 2049, 5001])
def test_append_and_gather_prompts(code, n):
    H, hd = 2, 128
    g = gen(n)
    n_pages = -(-n // 16) + 2
    pages = torch.randperm(n_pages, generator=g)[: -(-n // 16)]
    slots = (pages[torch.arange(n) // 16] * 16 + torch.arange(n) % 16).int()
    fused = torch.randn(n, 3 * H * hd + 8, generator=g).to(torch.bfloat16)
    k, v = fused[:, 8:8 + H * hd].view(n, H, hd), fused[:, 8 + 2 * H * hd:].view(n, H, hd)
    pool = np.full((n_pages, H, og.block_bytes(hd)), 0xFF, np.uint8)
    dev = to(DEV, pool)
    og.append(pool, k.float().numpy(), v.float().numpy(), slots.numpy(), code)
    fd = fused.to(DEV)
    bc.kv8_append(fd[:, 8:8 + H * hd].view(n, H, hd), fd[:, 8 + 2 * H * hd:].view(n, H, hd), slots.to(DEV), dev, code)
    torch.cuda.synchronize()
    blocks_equal(dev.cpu().numpy(), pool, hd)
    # read back: in order, shuffled, repeated, outside the pool
    some = torch.randint(0, n, (n,), generator=g)
    for sl in (slots, slots.flip(0), slots[some], torch.tensor([-1, n_pages * 16, int(slots[0]), -2 ** 31], dtype=torch.int32)):
        rk, rv = og.read(pool, sl.numpy(), code, hd)
        for dt in DTYPES:
            ko = torch.full((sl.numel(), H, hd), float("nan"), dtype=dt, device=DEV)
            vo = ko.clone()
            bc.kv8_gather(dev, sl.to(DEV), ko, vo, code)
            torch.cuda.synchronize()
            # code times scale is one f32 rounding of the product, then the type's
            for got, ref in ((ko, rk), (vo, rv)):
                ref32 = torch.from_numpy(ref).float()
                assert torch.equal(got.cpu(), ref32.to(dt))


@pytest.mark.parametrize("code", CODES)
def test_append_poisons_only_its_block(code):
    H, hd = 2, 64
    pool = make_pool(3, H, hd, code, seed=1)
    dev = to(DEV, pool)
    k = torch.zeros(2, H, hd)
    v = torch.zeros(2, H, hd)
    k[1, 1, 5] = float("inf")
    v[0, 0, 3] = float("nan")
    bc.kv8_append(k.to(DEV), v.to(DEV), ints([16, 17]), dev, code)
    got = dev.cpu().numpy()
    s = got[:, :, 32 * hd:32 * hd + 8].copy().view(np.float32)
    assert np.isnan(s[1, 1, 0]) and s[1, 0, 0] == 0 and np.isnan(s[1, 0, 1]) and s[1, 1, 1] == 0
    blocks_equal(got[[0, 2]], pool[[0, 2]], hd)
    # the page's next first token starts afresh
    bc.kv8_append(k[:1].to(DEV), torch.ones(1, H, hd, device=DEV), ints([16]), dev, code)
    s = dev.cpu().numpy()[:, :, 32 * hd:32 * hd + 8].copy().view(np.float32)
    assert np.isfinite(s).all()


# ------------------------------------------------------------------ attention
def run_attention(c, seed=0, poison=True):
    """One call against the definition.  c: lens, H, G, hd, code, dtype and options."""
    lens, H, G, hd, code, dtype = c["lens"], c["H"], c["G"], c["hd"], c["code"], c["dtype"]
    g = gen(seed + sum(lens) + hd)
    rng = np.random.default_rng(seed)
    B = len(lens)
    blocks = [og.pages_of(n) for n in lens]
    n_pages = sum(blocks) + 2
    pool = make_pool(n_pages, H, hd, code, seed=seed + 3)
    perm = rng.permutation(n_pages).astype(np.int32)
    max_blocks = max(max(blocks), 1) + c.get("extra_blocks", 1)
    table = np.full((B, max_blocks), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :blocks[b]] = perm[at:at + blocks[b]]
        at += blocks[b]
    if poison:
        # bytes that no row sees: the tokens behind a sequence's end, and the pages of nobody
        kp, vp = og._places(hd)
        for b in range(B):
            if lens[b] % 16:
                blk = pool[table[b, blocks[b] - 1]]
                blk[:, kp[lens[b] % 16:].ravel()] = 0x7F
                blk[:, vp[lens[b] % 16:].ravel()] = 0xFF
        pool[perm[at:]] = 0xFF
    for b, j in c.get("holes", []):
        table[b, j] = (-1, n_pages, 2 ** 30)[(b + j) % 3]
    qlens = c.get("qlens")
    q_start = None
    n_q = B
    max_q = 1
    if qlens is not None:
        q_start = np.cumsum([c.get("row0", 0)] + list(qlens)).astype(np.int32)
        n_q = int(q_start[-1]) + c.get("extra_rows", 0)
        max_q = c.get("max_q", max(qlens))
    width = H * G * hd
    pad = c.get("pad", 0)
    fused = (torch.randn(max(n_q, 1), width + pad, generator=g) * c.get("q_amp", 1.0)).to(dtype)
    q = fused[:n_q, :width].view(n_q, H * G, hd)
    pages = n_sel = None
    if c.get("keep"):
        K = max(1, int(max(blocks) * c["keep"]))
        pages = np.full((B, H, K + 1), 2 ** 30, np.int32)
        n_sel = np.zeros(B, np.int32)
        for b in range(B):
            n_sel[b] = min(K, blocks[b])
            for h in range(H):
                pages[b, h, :n_sel[b]] = np.sort(rng.permutation(blocks[b])[:n_sel[b]])
    slopes = np.exp2(-np.arange(1, H * G + 1) * 8.0 / (H * G)).astype(np.float32) if c.get("slopes") else None
    opt = dict(cap=c.get("cap", 0.0), window=c.get("window", 0))
    want = og.attention(q.float().numpy(), pool, lens, table, code, hd, q_start, max_q, pages, n_sel,
                        c.get("scale"), slopes=slopes, **opt)
    out = torch.full((n_q, H * G, hd), -77.0, dtype=dtype, device=DEV)
    scratch = torch.zeros(bc.bc_kv8_attention_scratch_bytes(B, H, G, max_q, hd), dtype=torch.uint8, device=DEV)
    fd = fused.to(DEV)
    args = (fd[:n_q, :width].view(n_q, H * G, hd), to(DEV, pool), ints(lens), ints(table), out, scratch, code)
    kw = dict(q_start=ints(q_start) if q_start is not None else None, max_q=max_q,
              pages=ints(pages) if pages is not None else None, n_sel=ints(n_sel) if n_sel is not None else None,
              scale=c.get("scale"), slopes=to(DEV, slopes) if slopes is not None else None, **opt)
    bc.kv8_attention(*args, **kw)
    torch.cuda.synchronize()
    assert bc.bc_kv8_attention_status(scratch.data_ptr(), None) == bc.BC_OK
    got = out.float().cpu().double().numpy()
    untouched = np.isnan(want)
    assert (got[untouched] == -77.0).all()
    live = pool[[int(p) for b in range(B) for p in table[b, :blocks[b]] if 0 <= p < n_pages]] if sum(blocks) else pool[:1] * 0
    tol = attention_tol(np.nan_to_num(want), q.float().numpy().astype(np.float64), live, code, hd, max(max(lens), 1), opt["cap"], slopes,
                        dtype == torch.bfloat16) if live.size else 0.0
    bad = ~untouched & ~(np.abs(got - want) <= tol)
    assert not bad.any(), (int(bad.sum()), float(np.nanmax(np.abs(got - want))), float(np.max(tol)))
    first = out.clone()
    for _ in range(2):
        out.fill_(-77.0)
        bc.kv8_attention(*args, **kw)
        torch.cuda.synchronize()
        assert torch.equal(out, first)                    # the same bits again, over the same scratch
    return got


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("lens", [[1], [16], [17], [5, 0, 300], [2049], [31, 1, 0, 700, 64, 3, 16]])
def test_attention_lengths(code, dtype, hd, lens):
    run_attention(dict(lens=lens, H=2, G=4, hd=hd, code=code, dtype=dtype))


@pytest.mark.parametrize("H,G", [(1, 1), (8, 8), (3, 5), (5, 7), (4, 2)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_attention_heads(H, G, dtype):
    run_attention(dict(lens=[70, 129, 1], H=H, G=G, hd=128, code="e4m3", dtype=dtype, pad=64))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("G,qlens", [(1, [3, 1, 2]), (4, [4, 4, 1]), (8, [8, 3, 0]), (3, [5, 2, 7]), (2, [32, 9, 1]),
                                     (1, [64, 64, 2])])
@pytest.mark.parametrize("hd", [64, 128])
def test_attention_several_queries(G, qlens, dtype, hd):
    run_attention(dict(lens=[200, 40, 7], H=2, G=G, hd=hd, code="int8", dtype=dtype, qlens=qlens, row0=2,
                       extra_rows=3))


@pytest.mark.parametrize("opt", [dict(cap=5.0), dict(window=1), dict(window=20), dict(window=400), dict(slopes=True),
                                 dict(cap=30.0, window=33, slopes=True), dict(keep=0.4), dict(keep=0.3, window=64),
                                 dict(scale=0.3), dict(scale=-0.1), dict(scale=0.0), dict(q_amp=1e-20), dict(keep=1.0, cap=2.0)])
@pytest.mark.parametrize("code,dtype", [("e4m3", torch.float32), ("int8", torch.bfloat16)])
def test_attention_options(opt, code, dtype):
    run_attention(dict(lens=[333, 12, 0, 180], H=2, G=4, hd=128, code=code, dtype=dtype, qlens=[2, 1, 1, 3], **opt))
    run_attention(dict(lens=[333, 12, 0, 180], H=2, G=4, hd=64, code=code, dtype=dtype, **opt))


def test_attention_rows_that_see_nothing():
    # more queries than tokens; a list that keeps only pages behind a row's window; pages that are not there
    got = run_attention(dict(lens=[2, 40], H=1, G=2, hd=64, code="e4m3", dtype=torch.float32, qlens=[4, 1]))
    assert (got[:2] == 0).all()
    got = run_attention(dict(lens=[500], H=2, G=2, hd=64, code="int8", dtype=torch.float32, keep=0.05, window=1))
    got = run_attention(dict(lens=[40, 33], H=1, G=2, hd=64, code="e4m3", dtype=torch.float32,
                             holes=[(0, 0), (0, 1), (0, 2), (1, 1)]))
    assert (got[0] == 0).all() and (got[1] != 0).all()


def test_attention_more_queries_than_max_q():
    run_attention(dict(lens=[100, 50], H=1, G=4, hd=64, code="e4m3", dtype=torch.bfloat16, qlens=[6, 2], max_q=3))


@pytest.mark.parametrize("B", [200, 2048])
def test_attention_many_sequences(B):
    rng = np.random.default_rng(B)
    lens = [int(x) for x in rng.integers(0, 60, B)]
    run_attention(dict(lens=lens, H=1, G=2, hd=64, code="int8", dtype=torch.bfloat16))


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dtype,qlens", [(torch.float32, [1, 1]), (torch.bfloat16, [4, 2])])
def test_attention_long(code, dtype, qlens):
    run_attention(dict(lens=[40000, 777], H=2, G=4, hd=128, code=code, dtype=dtype, qlens=qlens))


def test_attention_lengths_beyond_the_table():
    # 500 tokens claimed, a table of 2 + 1 blocks: taken as 48
    c = dict(lens=[30], H=1, G=2, hd=64, code="e4m3", dtype=torch.float32)
    pool = make_pool(4, 1, 64, "e4m3", seed=9)
    table = np.array([[2, 0, 1]], np.int32)
    q = torch.randn(1, 2, 64, generator=gen(1))
    out = torch.empty(1, 2, 64, device=DEV)
    scratch = torch.zeros(bc.bc_kv8_attention_scratch_bytes(1, 1, 2, 1, 64), dtype=torch.uint8, device=DEV)
    for n, eff in ((500, 48), (2 ** 31 - 1, 48), (-3, 0)):
        want = og.attention(q.numpy(), pool, [eff], table, "e4m3", 64)
        bc.kv8_attention(q.to(DEV), to(DEV, pool), ints([n]), ints(table), out, scratch, c["code"])
        tol = attention_tol(want, q.numpy().astype(np.float64), pool, "e4m3", 64, 48, 0.0, None, False)
        assert (np.abs(out.cpu().double().numpy() - want) <= tol).all()


@pytest.mark.parametrize("code", CODES)
def test_attention_unequal_value_scales(code):
    """Value scales many orders of magnitude apart, a page of zeros, and a
    page whose keys or values are not numbers where nobody looks."""
    H, G, hd, n = 1, 2, 64, 6 * 16
    g = gen(4)
    k = torch.randn(n, H, hd, generator=g).numpy()
    v = torch.randn(n, H, hd, generator=g).numpy()
    for p, f in enumerate([1e-30, 1e30, 0.0, 1e-6, 1.0, 1e3]):
        v[p * 16:(p + 1) * 16] *= f
    pool = np.zeros((7, H, og.block_bytes(hd)), np.uint8)
    og.append(pool, k, v, np.arange(n), code)
    table = np.arange(6, dtype=np.int32)[None]
    q = torch.randn(1, G, hd, generator=g)
    scratch = torch.zeros(bc.bc_kv8_attention_scratch_bytes(1, H, G, 1, hd), dtype=torch.uint8, device=DEV)
    out = torch.empty(1, G, hd, device=DEV)
    for keep in ([0], [2], [0, 2], [3, 4], [0, 3], [0, 1, 2, 3, 4, 5], [5, 4]):
        keep = sorted(keep)
        pages, n_sel = np.array([[keep]], np.int32), np.array([len(keep)], np.int32)
        want = og.attention(q.numpy(), pool, [n], table, code, hd, pages=pages, n_sel=n_sel)
        bc.kv8_attention(q.to(DEV), to(DEV, pool), ints([n]), ints(table), out, scratch, code, pages=ints(pages), n_sel=ints(n_sel))
        got = out.cpu().double().numpy()
        tol = attention_tol(want, q.numpy().astype(np.float64), pool[keep], code, hd, n, 0.0, None, False)
        assert (np.abs(got - want) <= tol).all(), keep


@pytest.mark.parametrize("dtype", DTYPES)
def test_attention_value_scale_not_a_number(dtype):
    """It makes every row that sees the block not a number, whatever the weight
    and the codes: one token of positive codes, or a weight that is 0 (of
    sequences so many that a warp reads both pages of some)."""
    hd, B = 64, 2000
    k = np.zeros((32, 1, hd), np.float32)
    k[:16, 0, 0] = 8.0
    v = np.ones((32, 1, hd), np.float32)
    pool = np.zeros((2, 1, og.block_bytes(hd)), np.uint8)
    og.append(pool, k, v, np.arange(32), "e4m3")
    pool[1, 0, 32 * hd + 4:32 * hd + 8] = np.array([np.nan], np.float32).view(np.uint8)
    q = torch.zeros(B, 1, hd, dtype=dtype)
    q[1:, 0, 0] = 8000.0               # the logits of page 0 are 8000 above those of page 1
    out = torch.empty(B, 1, hd, dtype=dtype, device=DEV)
    scratch = torch.zeros(bc.bc_kv8_attention_scratch_bytes(B, 1, 1, 1, hd), dtype=torch.uint8, device=DEV)
    bc.kv8_attention(q.to(DEV), to(DEV, pool), ints([1] + [32] * (B - 1)), ints([[1, 0]] + [[0, 1]] * (B - 1)), out,
                     scratch, "e4m3")
    assert torch.isnan(out).all()


def test_attention_lists_without_pages():
    """A list of no pages sees nothing; one that could hold none is refused
    (an empty tensor has no address, which would mean every page)."""
    pool, q, out = to(DEV, make_pool(4, 1, 64, "int8", seed=1)), torch.randn(2, 2, 64, generator=gen(1)).to(DEV), \
        torch.full((2, 2, 64), 7.0, device=DEV)
    scratch = torch.zeros(bc.bc_kv8_attention_scratch_bytes(2, 1, 2, 1, 64), dtype=torch.uint8, device=DEV)
    call = lambda pages: bc.kv8_attention(q, pool, ints([20, 40]), ints([[0, 1, 2], [1, 2, 3]]), out, scratch, "int8",
                                          pages=pages, n_sel=ints([0, 0]))
    with pytest.raises(ValueError, match="max_sel"):
        call(torch.zeros(2, 1, 0, dtype=torch.int32, device=DEV))
    assert (out == 7).all()
    call(torch.zeros(2, 1, 3, dtype=torch.int32, device=DEV))
    assert (out == 0).all()


def test_attention_not_a_number():
    """A poisoned block reaches the rows of its head that see it, no others."""
    H, G, hd = 2, 2, 64
    pool = make_pool(4, H, hd, "e4m3", seed=2)
    pool[1, 0, 32 * hd:32 * hd + 4] = np.array([np.nan], np.float32).view(np.uint8)
    pool[2, 1, 32 * hd + 4:32 * hd + 8] = np.array([np.nan], np.float32).view(np.uint8)
    table = np.array([[0, 1, 3, 3], [0, 3, 2, 3], [3, 0, 3, 3]], np.int32)
    q = torch.randn(3, H * G, hd, generator=gen(3))
    q[2, 3, 5] = float("inf")
    q[2, 1, 0] = float("nan")
    scratch = torch.zeros(bc.bc_kv8_attention_scratch_bytes(3, H, G, 1, hd), dtype=torch.uint8, device=DEV)
    out = torch.empty(3, H * G, hd, device=DEV)
    bc.kv8_attention(q.to(DEV), to(DEV, pool), ints([40, 48, 40]), ints(table), out, scratch, "e4m3")
    nan = torch.isnan(out).all(-1).cpu().numpy()
    fine = torch.isfinite(out).all(-1).cpu().numpy()
    want = np.array([[1, 1, 0, 0], [0, 0, 1, 1], [0, 1, 0, 1]], bool)
    assert (nan == want).all() and (fine == ~want).all()
    # behind a window of 8 the poisoned page is not seen
    bc.kv8_attention(q[:1].to(DEV), to(DEV, pool), ints([40]), ints(table[:1]), out[:1], scratch, "e4m3", window=8)
    assert torch.isfinite(out[0]).all()


# ------------------------------------------------------------------ logits
def run_logits(B, V, dtype, seed, hist=None, bias=0, masks=0, rows=False, pads=False, prompt=True, pen=(1, 1, 1),
               in_place=False, stride=0):
    rng = np.random.default_rng(seed)
    wide = torch.from_numpy(rng.standard_normal((B, V + stride)).astype(np.float32) * 3).to(dtype)
    wide[0, 0] = float("inf")
    if V > 3:
        wide[0, 1], wide[0, 2], wide[0, 3] = float("-inf"), float("nan"), 0.0
    x = wide[:, :V]
    kw = {}
    if hist is not None:
        n = rng.integers(0, hist + 1, B)
        kw["hist_start"] = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        h = np.minimum(rng.integers(0, V, n.sum()), rng.integers(0, V, n.sum()))
        if pads and len(h):
            h[::3] = rng.choice([-1, V, V + 5, -2 ** 31, 2 ** 31 - 1], len(h[::3]))
        kw["hist"] = h.astype(np.int32)
        if prompt:
            kw["prompt_len"] = rng.integers(-1, hist + 2, B).astype(np.int32)
    for on, name, lo in zip(pen, ("repetition", "frequency", "presence"), (0.7, -0.5, -0.5)):
        if on:
            kw[name] = (lo + rng.random(B)).astype(np.float32)
    if bias:
        ids = rng.integers(-1, min(V, 40) + 1, B * bias)             # many ids twice, some outside
        kw["bias_ids"], kw["bias_vals"] = ids.astype(np.int32), (5 * rng.standard_normal(B * bias)).astype(np.float32)
        kw["bias_start"] = (np.arange(B + 1) * bias).astype(np.int32)
    if masks:
        kw["mask"] = rng.integers(-2 ** 31, 2 ** 31, (masks, -(-V // 32))).astype(np.int32)
        kw["mask"][0] = 0                                            # a mask that leaves nothing
        if rows:
            kw["mask_row"] = rng.integers(-2, masks + 2, B).astype(np.int32)
    want = og.logits_adjust(x.double().numpy(), **kw)
    src = wide.to(DEV)[:, :V]
    out = src if in_place else torch.full((B, V), 77.0, dtype=dtype, device=DEV)
    bc.logits_adjust(src, out, **{k: to(DEV, v) for k, v in kw.items()})
    torch.cuda.synchronize()
    got = out.double().cpu().numpy()
    np.testing.assert_array_equal(np.isnan(got), np.isnan(want))
    np.testing.assert_array_equal(np.isinf(got), np.isinf(want))
    np.testing.assert_array_equal(got[np.isinf(want)], want[np.isinf(want)])
    # at most five f32 roundings, of values no larger than |x| r + |f c| + |p| + |bias|, then the output's
    big = np.abs(x.double().numpy()) * 2 + (1.5 * ((hist or 0) + 1)) + 25.0
    tol = 5 * 2.0 ** -24 * big + (np.abs(want) * 2.0 ** -8 if dtype == torch.bfloat16 else 0.0)
    ok = np.isfinite(want)
    assert (np.abs(got[ok] - want[ok]) <= tol[ok]).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,V", [(1, 1), (1, 5), (3, 31), (2, 33), (5, 4096), (2, 4097), (1, 32001), (3, 128256)])
def test_logits_all(B, V, dtype):
    run_logits(B, V, dtype, seed=V + B, hist=50, bias=7, masks=B, pads=True)
    run_logits(B, V, dtype, seed=V + B + 1, hist=50, bias=7, masks=3, rows=True, in_place=True)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kw", [dict(), dict(hist=20), dict(hist=20, prompt=False), dict(hist=20, pen=(1, 0, 0)),
                                dict(hist=20, pen=(0, 1, 0)), dict(hist=20, pen=(0, 0, 1)), dict(hist=20, pen=(0, 0, 0)),
                                dict(bias=90), dict(masks=2, rows=True), dict(masks=4), dict(hist=0, bias=1),
                                dict(hist=5000, bias=3), dict(hist=9, stride=3, bias=2, masks=4)])
def test_logits_parts(kw, dtype):
    run_logits(4, 1500, dtype, seed=7, **kw)
    run_logits(4, 1501, dtype, seed=8, in_place=True, **kw)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V,at,pad,at_out,pad_out", [(1, 3, 1, 0, 0), (2, 1, 3, 1, 3), (7, 7, 6, 2, 1), (8, 5, 0, 5, 0),
                                                     (9, 1, 8, 1, 0), (2047, 2, 1, 6, 3), (4095, 1, 1, 3, 7),
                                                     (8185, 7, 5, 7, 5), (8192, 3, 1, 0, 0), (8193, 0, 2, 4, 1),
                                                     (20001, 6, 1, 2, 2)])
def test_logits_rows_anywhere(V, at, pad, at_out, pad_out, dtype):
    """Rows that begin at any multiple of their type, other ones in than out,
    and nothing written beside them."""
    B, rng = 5, np.random.default_rng(V)
    make = lambda off, stride: torch.full((off + B * stride + 16,), 77.0, dtype=dtype, device=DEV)
    view = lambda buf, off, stride: buf[off:off + B * stride].view(B, stride)[:, :V]
    src, dst = make(at, V + pad), make(at_out, V + pad_out)
    x, out = view(src, at, V + pad), view(dst, at_out, V + pad_out)
    x.copy_(torch.from_numpy(rng.standard_normal((B, V)).astype(np.float32)))
    n = 40
    kw = dict(hist=rng.integers(0, V, B * n), hist_start=np.arange(B + 1) * n, prompt_len=np.arange(B) * 9,
              bias_ids=rng.integers(0, V, B * 6), bias_start=np.arange(B + 1) * 6,
              mask=rng.integers(-2 ** 31, 2 ** 31, (B, -(-V // 32))))
    kw = {k: v.astype(np.int32) for k, v in kw.items()}
    kw.update(bias_vals=rng.standard_normal(B * 6).astype(np.float32), repetition=np.float32([1.3, 0.8, 1, 2, 0.5]),
              frequency=np.float32([0.2, 0, -0.1, 0.3, 0.1]), presence=np.float32([0, 0.2, 0.1, -0.3, 0.4]))
    want = og.logits_adjust(x.double().cpu().numpy(), **kw)
    # as in run_logits: five f32 roundings of values below 2 |x| + 0.3 * 40 + 0.4 + |bias|, |x| and |bias| below 8
    tol = 5 * 2.0 ** -24 * 40 + (np.abs(want) * 2.0 ** -8 if dtype == torch.bfloat16 else 0.0)
    dev = {k: to(DEV, v) for k, v in kw.items()}
    for o, buf, off, stride in ((out, dst, at_out, V + pad_out), (x, src, at, V + pad)):       # then in place
        bc.logits_adjust(x, o, **dev)
        got, ok = o.double().cpu().numpy(), np.isfinite(want)
        np.testing.assert_array_equal(got[~ok], want[~ok])
        assert (np.abs(got[ok] - want[ok]) <= np.broadcast_to(tol, want.shape)[ok]).all()
        rest = torch.ones_like(buf, dtype=torch.bool)
        view(rest, off, stride)[:] = False
        assert (buf[rest] == 77).all()


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("code,dtype", [("e4m3", torch.bfloat16), ("int8", torch.float32)])
@pytest.mark.parametrize("graph", [False, True])
def test_a_ragged_run(code, dtype, graph):
    """Prompts of different lengths enter, sequences decode, drafts are
    taken back, one leaves and another takes its pages: the cache's content
    and every attention against the definition on the same inputs."""
    L, B, H, G, hd, max_q = 2, 5, 2, 4, 64, 4
    n_pages, max_blocks, max_tokens = 24, 8, 120
    cache = bc.RaggedCache(L, B, n_pages, H, G, hd, max_blocks, max_tokens, max_q, code, device=DEV)
    rng = np.random.default_rng(3)
    lens = np.zeros(B, np.int32)
    table, free, n_free = np.zeros((B, max_blocks), np.int32), np.arange(n_pages, dtype=np.int32), n_pages
    pool = np.zeros((L, n_pages, H, og.block_bytes(hd)), np.uint8)
    steps = [[33, 0, 17, 50, 0], [1, 16, 1, 1, 0], [4, 2, 4, 1, 0], [-2, 0, -4, 1, 3], [1, 1, 1, -1000, 60],
             [1, 1, 1, 40, 1], [3, 1, 2, 1, 4]]
    delta_d = ints(np.zeros(B))
    kd = [torch.zeros(max_tokens, H, hd, dtype=dtype, device=DEV) for _ in range(2 * L)]
    qd = torch.zeros(max_tokens, H * G, hd, dtype=dtype, device=DEV)
    outs = [torch.zeros(max_tokens, H * G, hd, dtype=dtype, device=DEV) for _ in range(L)]

    def step():
        cache.plan(delta_d)
        for l in range(L):
            cache.append(l, kd[2 * l], kd[2 * l + 1])
            cache.attend(l, qd, outs[l], window=40, cap=20.0)

    captured = None
    if graph:
        step()                                           # kernels set up outside the capture
        torch.cuda.synchronize()
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            step()
    for delta in steps:
        delta = np.array(delta, np.int32)
        k = [torch.from_numpy(rng.standard_normal((max_tokens, H, hd)).astype(np.float32)).to(dtype) for _ in range(2 * L)]
        q = torch.from_numpy(rng.standard_normal((max_tokens, H * G, hd)).astype(np.float32)).to(dtype)
        delta_d.copy_(ints(delta))
        for d, s in zip(kd + [qd], k + [q]):
            d.copy_(s)
        for o in outs:
            o.fill_(-77.0)
        captured.replay() if graph else step()
        torch.cuda.synchronize()
        w = og.block_tables(lens, delta, table, free, n_free, max_tokens)
        lens, table, free, n_free = w["lens"], w["table"], w["free_list"], w["n_free"]
        np.testing.assert_array_equal(cache.lens.cpu().numpy(), lens)
        np.testing.assert_array_equal(cache.table.cpu().numpy(), table)
        np.testing.assert_array_equal(cache.slots.cpu().numpy(), w["slots"])
        assert int(cache.n_free) == n_free
        for l in range(L):
            og.append(pool[l], k[2 * l].float().numpy(), k[2 * l + 1].float().numpy(), w["slots"], code)
            blocks = cache.pool[l].cpu().numpy()
            for b in range(B):
                for p in table[b, :og.pages_of(lens[b])]:
                    blocks_equal(blocks[p], pool[l][p], hd)
            want = og.attention(q.float().numpy(), pool[l], lens, table, code, hd, w["q_start"], max_q, window=40, cap=20.0)
            got = outs[l].float().cpu().double().numpy()
            none = np.isnan(want)
            assert (got[none] == -77.0).all()
            used = pool[l][[int(p) for b in range(B) for p in table[b, :og.pages_of(lens[b])]]]
            tol = attention_tol(np.nan_to_num(want), q.float().numpy().astype(np.float64), used, code, hd, int(lens.max()), 20.0, None,
                                dtype == torch.bfloat16)
            assert (np.abs(got - want)[~none] <= tol[~none] if np.ndim(tol) else tol).all()
    cache.status()
    # a prefix read back into a decode model's cache
    n = int(lens[0])
    k, v = cache.read(0, 0, n)
    rk, rv = og.read(pool[0], w_slots(table, 0, n), code, hd)
    assert torch.equal(k.cpu(), torch.from_numpy(rk).float().to(torch.bfloat16))
    assert torch.equal(v.cpu(), torch.from_numpy(rv).float().to(torch.bfloat16))


def w_slots(table, b, n):
    return [int(table[b, t // 16]) * 16 + t % 16 for t in range(n)]


def test_model_logits_and_prefix():
    """The 8-bit cache's prefix continues in a Model, whose step's logits are
    adjusted in place: the model's own step over the same (decoded) prefix."""
    from synth import TINY, make_weights
    cfg = TINY
    L, H, hd = cfg["n_layers"], cfg["n_kv_heads"], cfg["head_dim"]
    w = {k: t.to(DEV) for k, t in make_weights(cfg, seed=0).items()}
    n = 75
    cache = bc.RaggedCache(L, 1, 8, H, cfg["n_heads"] // H, hd, 8, 128, code="int8", device=DEV)
    cache.plan(ints([n]))
    g = gen(8)
    kv = [torch.randn(n, H, hd, generator=g).to(DEV) for _ in range(2 * L)]
    for l in range(L):
        cache.append(l, kv[2 * l], kv[2 * l + 1])
    parts = [cache.read(l, 0, n) for l in range(L)]
    k = torch.stack([p[0] for p in parts]).transpose(1, 2).contiguous()
    v = torch.stack([p[1] for p in parts]).transpose(1, 2).contiguous()
    m = bc.Model(cfg, w, n + 8)
    m.append(k, v)
    logits = torch.empty(1, cfg["vocab"], device=DEV)
    m.step(17, "dense", logits[0])
    before = logits.clone()
    hist = ints([17, 5, 17, 9])
    bc.logits_adjust(logits, logits, hist=hist, hist_start=ints([0, 4]), repetition=torch.full((1,), 1.2, device=DEV),
                     frequency=torch.full((1,), 0.3, device=DEV), presence=torch.full((1,), 0.1, device=DEV))
    want = og.logits_adjust(before.cpu().double().numpy(), hist.cpu().numpy(), np.array([0, 4]),
                            repetition=np.float32([1.2]), frequency=np.float32([0.3]), presence=np.float32([0.1]))
    assert np.abs(logits.cpu().double().numpy() - want).max() <= 5 * 2.0 ** -24 * (2 * before.abs().max().item() + 2)
    m.close()


def test_other_streams():
    s = torch.cuda.Stream()
    H, hd = 2, 64
    pool = torch.zeros(4, H, og.block_bytes(hd), dtype=torch.uint8, device=DEV)
    k = torch.randn(20, H, hd, device=DEV)
    slots = ints(range(20))
    ko, vo = torch.empty_like(k), torch.empty_like(k)
    torch.cuda.synchronize()
    bc.kv8_append(k, k, slots, pool, "int8", stream=s)
    bc.kv8_gather(pool, slots, ko, vo, "int8", stream=s)
    s.synchronize()
    top = k.abs().amax().item()
    assert (ko - k).abs().max().item() <= top / 127 / 2 * 1.01 and torch.equal(ko, vo)


@pytest.mark.parametrize("hist,bias", [(30000, 0), (30000, 2), (12288, 0), (12286, 2), (12287, 2), (3, 13000)])
def test_logits_long_lists(hist, bias):
    """Histories and bias lists on both sides of what a hash table takes, with
    more distinct ids than it has room for."""
    V, g = 40000, gen(hist + bias)
    x = torch.randn(2, V, generator=g)
    h = torch.cat([torch.randperm(V, generator=g)[:hist], torch.randperm(V, generator=g)[: hist // 2]]).int()
    hs = np.array([0, hist, hist + hist // 2], np.int32)
    kw = dict(hist=h.numpy(), hist_start=hs, prompt_len=np.array([hist // 3, 0], np.int32),
              repetition=np.float32([1.3, 0.8]), frequency=np.float32([0.2, -0.1]), presence=np.float32([0.1, 0.4]))
    if bias:
        kw.update(bias_ids=torch.randint(0, V, (2 * bias,), generator=g).int().numpy(),
                  bias_vals=torch.randn(2 * bias, generator=g).numpy(), bias_start=np.array([0, bias, 2 * bias], np.int32))
    want = og.logits_adjust(x.double().numpy(), **kw)
    for out in (torch.full((2, V), 77.0, device=DEV), None):
        src = x.to(DEV)
        out = src if out is None else out
        bc.logits_adjust(src, out, **{k: to(DEV, v) for k, v in kw.items()})
        assert np.abs(out.cpu().double().numpy() - want).max() <= 5 * 2.0 ** -24 * 20


def attention_inputs(lens, H, G, hd, code, seed=0):
    """(q, pool, lens, table, definition) of one query a sequence."""
    blocks = [og.pages_of(n) for n in lens]
    pool = make_pool(sum(blocks) + 1, H, hd, code, seed=seed)
    table = np.full((len(lens), max(blocks) + 1), -1, np.int32)
    at = 0
    for b, n in enumerate(blocks):
        table[b, :n] = np.arange(at, at + n)[::-1]
        at += n
    q = torch.randn(len(lens), H * G, hd, generator=gen(seed + 1))
    want = og.attention(q.numpy(), pool, lens, table, code, hd)
    tol = attention_tol(want, q.double().numpy(), pool, code, hd, max(lens), 0.0, None, False)
    return q.to(DEV), to(DEV, pool), ints(lens), ints(table), want, tol


def test_attention_calls_of_any_sizes_share_a_scratch():
    cases = [([3000], 1, 8, 64, "int8"), ([700, 90, 16] * 5, 3, 2, 128, "e4m3"), ([5], 1, 1, 64, "e4m3"),
             ([2000, 1, 400], 4, 8, 128, "int8")]
    need = max(bc.bc_kv8_attention_scratch_bytes(len(l), H, G, 1, hd) for l, H, G, hd, _ in cases)
    scratch = torch.zeros(need, dtype=torch.uint8, device=DEV)
    made = [(c, attention_inputs(*c, seed=i)) for i, c in enumerate(cases)]
    for _ in range(2):
        for (lens, H, G, hd, code), (q, pool, ld, table, want, tol) in made:
            out = torch.empty_like(q)
            bc.kv8_attention(q, pool, ld, table, out, scratch, code)
            assert (np.abs(out.cpu().double().numpy() - want) <= tol).all()


def test_two_streams_at_once():
    """Calls that overlap, each with a scratch of its own, and a plan beside them."""
    made = [attention_inputs([2500, 30, 700], 2, 4, 128, "e4m3", seed=i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    scratch = [torch.zeros(bc.bc_kv8_attention_scratch_bytes(3, 2, 4, 1, 128), dtype=torch.uint8, device=DEV) for _ in range(2)]
    outs = [[torch.empty_like(m[0]) for _ in range(20)] for m in made]
    torch.cuda.synchronize()
    for i in range(20):
        for s in range(2):
            q, pool, ld, table, _, _ = made[s]
            bc.kv8_attention(q, pool, ld, table, outs[s][i], scratch[s], "e4m3", stream=streams[s])
    torch.cuda.synchronize()
    for s in range(2):
        for o in outs[s]:
            assert torch.equal(o, outs[s][0])
        assert (np.abs(outs[s][0].cpu().double().numpy() - made[s][4]) <= made[s][5]).all()


def test_wrappers_say_what_is_wrong():
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device=DEV)
    f = lambda *s, **k: torch.zeros(*s, device=DEV, **k)
    pool = torch.zeros(4, 2, 32 * 64 + 32, dtype=torch.uint8, device=DEV)
    x = f(3, 2, 64)

    def refused(what, fn, *args, **kw):
        with pytest.raises(ValueError, match=what):
            fn(*args, **kw)

    for bad in (i(3).long(), i(6)[::2], i(3).cpu(), i(2)):
        refused("slots|k must be", bc.kv8_append, x, x, bad, pool)
        refused("slots|k_out must be", bc.kv8_gather, pool, bad, x, x)
    refused("v must be", bc.kv8_append, x, x.to(torch.bfloat16), i(3), pool)
    refused("float32 or bfloat16", bc.kv8_append, x.half(), x.half(), i(3), pool)
    refused("k must be", bc.kv8_append, f(3, 64, 2).transpose(1, 2).contiguous()[:, :, :63], x, i(3), pool)
    refused("dense", bc.kv8_append, f(3, 64, 2).transpose(1, 2), x, i(3), pool)
    refused("code", bc.kv8_append, x, x, i(3), pool, "fp4")
    refused("pool", bc.kv8_append, x, x, i(3), pool[:, :, :2000])
    refused("pool", bc.kv8_append, x, x, i(3), pool[::2])
    refused("contiguous", bc.kv8_gather, pool, i(3), f(6, 2, 64)[::2], x)
    sc = torch.zeros(1 << 20, dtype=torch.uint8, device=DEV)
    q, lens, table = f(3, 8, 64), i(3), i(3, 4)
    ok = lambda **k: bc.kv8_attention(**{**dict(q=q, pool=pool, lens=lens, table=table, out=f(3, 8, 64), scratch=sc), **k})
    ok()
    refused("lens", ok, lens=i(4))
    refused("table", ok, table=i(12))
    refused("table", ok, table=i(3, 4).float())
    refused("out", ok, out=f(3, 8, 64, dtype=torch.bfloat16))
    refused("out", ok, out=f(3, 8, 128)[:, :, ::2])
    refused("q must be", ok, q=f(3, 7, 64))
    refused("heads and dims of q", ok, q=f(3, 64, 8).transpose(1, 2))
    refused("one query row", ok, max_q=2)
    refused("q_start", ok, q_start=i(3), max_q=2)
    refused("go together", ok, pages=i(3, 2, 4))
    refused("pages must be", ok, pages=i(3, 1, 4), n_sel=i(3))
    refused("slopes", ok, slopes=f(7))
    refused("scratch", ok, scratch=sc.float())
    with pytest.raises(bc.BCError):
        ok(scratch=sc[:4096])                            # too small
    with pytest.raises(bc.BCError):
        ok(q=f(3 * 8 * 64 + 2)[2:].view(3, 8, 64))       # not 16-byte aligned
    with pytest.raises(bc.BCError):
        ok(q=f(3, 8 * 64 + 4)[:, :512].view(3, 8, 64))   # a row stride that is not a multiple of 8
    with pytest.raises(bc.BCError):
        ok(window=-1)
    with pytest.raises(bc.BCError):
        bc.kv8_append(f(3, 130)[:, :128].view(3, 2, 64), x, i(3), pool)
    lg = f(2, 50)
    refused("out must", bc.logits_adjust, lg, f(2, 51))
    refused("dense", bc.logits_adjust, f(50, 2).t(), lg)
    refused("go together", bc.logits_adjust, lg, lg, hist=i(3))
    refused("hist_start", bc.logits_adjust, lg, lg, hist=i(3), hist_start=i(2))
    refused("bias_vals", bc.logits_adjust, lg, lg, bias_ids=i(3), bias_vals=f(2), bias_start=i(3))
    refused("repetition", bc.logits_adjust, lg, lg, repetition=f(3))
    refused("mask must be", bc.logits_adjust, lg, lg, mask=i(2, 1))
    refused("mask_row", bc.logits_adjust, lg, lg, mask_row=i(2))
    with pytest.raises(bc.BCError):
        bc.logits_adjust(lg, lg, mask=i(1, 2))           # two rows, one mask
    t = dict(lens=i(2), delta=i(2), table=i(2, 3), free_list=i(5), n_free=i(1), lens_out=i(2), n_free_out=i(1),
             q_start=i(3), slots=i(4), positions=i(4), ticket=i(1))
    bc.block_tables(**t)
    for k, v in dict(lens=i(3), q_start=i(2), positions=i(3), n_free=i(2), delta=i(2).float(), free_list=i(10)[::2]).items():
        refused(k, bc.block_tables, **{**t, k: v})
    torch.cuda.synchronize()


# ------------------------------------------------------------------ beyond 32 bits
def test_a_pool_beyond_4_gib():
    """Pages whose bytes lie past 2^32 in the pool: the same bits as from a
    small pool."""
    H, G, hd, code = 8, 4, 128, "e4m3"
    block = og.block_bytes(hd)
    n_pages = 2 ** 32 // (H * block) + 40
    big = torch.empty(n_pages, H, block, dtype=torch.uint8, device=DEV)
    small = torch.zeros(12, H, block, dtype=torch.uint8, device=DEV)
    shift = n_pages - 12
    assert shift * H * block > 2 ** 32
    g = gen(5)
    n = 12 * 16 - 3
    k, v = (torch.randn(n, H, hd, generator=g).to(DEV) for _ in range(2))
    q = torch.randn(1, H * G, hd, generator=g).to(DEV)
    res = []
    for pool, first in ((small, 0), (big, shift)):
        pages = torch.arange(first, first + 12, device=DEV).flip(0).int()
        pos = torch.arange(n, device=DEV)
        slots = (pages[pos // 16] * 16 + pos % 16).int()
        bc.kv8_append(k, v, slots, pool, code)
        ko, vo = torch.empty_like(k), torch.empty_like(v)
        bc.kv8_gather(pool, slots, ko, vo, code)
        out = torch.empty_like(q)
        scratch = torch.zeros(bc.bc_kv8_attention_scratch_bytes(1, H, G, 1, hd), dtype=torch.uint8, device=DEV)
        bc.kv8_attention(q, pool, ints([n]), pages[None].contiguous(), out, scratch, code)
        res.append((ko, vo, out))
    for a, b in zip(*res):
        assert torch.equal(a, b)
    assert (res[0][0] - k).abs().max() < 0.07 * k.abs().max()


def test_outputs_beyond_2_31_elements():
    H, hd, n = 8, 128, 2 ** 31 // (8 * 128) + 50
    pool = to(DEV, make_pool(3, H, hd, "int8", seed=6))
    slots = (torch.arange(n, device=DEV) * 7 % 48).int()
    k = torch.empty(n, H, hd, dtype=torch.bfloat16, device=DEV)
    v = torch.empty_like(k)
    bc.kv8_gather(pool, slots, k, v, "int8")
    rk, rv = og.read(pool.cpu().numpy(), slots[-60:].cpu().numpy(), "int8", hd)
    assert torch.equal(k[-60:].cpu(), torch.from_numpy(rk).float().to(torch.bfloat16))
    assert torch.equal(v[-60:].cpu(), torch.from_numpy(rv).float().to(torch.bfloat16))
    del k, v
    B, V = 17000, 128256
    assert B * V > 2 ** 31
    x = torch.zeros(B, V, dtype=torch.bfloat16, device=DEV)
    x[-1] = 2.0
    hist = ints([5, V - 1, 5])
    starts = torch.zeros(B + 1, dtype=torch.int32, device=DEV)
    starts[-1] = 3
    bc.logits_adjust(x, x, hist=hist, hist_start=starts, repetition=torch.full((B,), 2.0, device=DEV),
                     frequency=torch.full((B,), 0.25, device=DEV))
    assert (x[:-1] == 0).all()
    want = torch.full((V,), 2.0)
    want[5], want[V - 1] = 0.5, 0.75
    assert torch.equal(x[-1].float().cpu(), want)


def test_wrappers_refuse_sizes_beyond_32_bits():
    """They would reach the C interface cut to their lower 32 bits."""
    pool, q = to(DEV, make_pool(2, 1, 64, "e4m3", seed=1)), torch.zeros(1, 1, 64, device=DEV)
    out = torch.full_like(q, 7.0)
    scratch = torch.zeros(bc.bc_kv8_attention_scratch_bytes(1, 1, 1, 1, 64), dtype=torch.uint8, device=DEV)
    for kw in (dict(window=2 ** 32 + 8), dict(window=-2 ** 32 + 8), dict(q_start=ints([0, 1]), max_q=2 ** 32 + 1)):
        with pytest.raises(ValueError, match="2\\^31"):
            bc.kv8_attention(q, pool, ints([20]), ints([[0, 1]]), out, scratch, "e4m3", **kw)
    lg = torch.full((1, 40), 7.0, device=DEV)
    if torch.cuda.mem_get_info()[0] > 24 << 30:
        with pytest.raises(ValueError, match="2\\^31"):
            bc.logits_adjust(lg, lg, hist=torch.empty(2 ** 32 + 4, dtype=torch.int32, device=DEV), hist_start=ints([0, 4]))
        torch.cuda.empty_cache()
    assert (out == 7).all() and (lg == 7).all()


@pytest.mark.parametrize("n_masks", [0, 1])
def test_logits_refuse_fewer_masks_than_rows(n_masks):
    lg = torch.full((2, 40), 7.0, device=DEV)
    with pytest.raises((ValueError, bc.BCError), match="mask for each|n_masks"):
        bc.logits_adjust(lg, lg, mask=torch.zeros(n_masks, 2, dtype=torch.int32, device=DEV))
    # with mask_row a row outside them has none
    bc.logits_adjust(lg, lg, mask=torch.zeros(n_masks, 2, dtype=torch.int32, device=DEV), mask_row=ints([n_masks, -1]))
    assert (lg == 7).all()


def test_read_stops_at_the_end_of_a_sequence():
    """Entries of the table behind a sequence's pages are old or zero: the
    pages of others."""
    c = bc.RaggedCache(1, 2, 8, 1, 1, 64, 4, 64, code="int8", device=DEV)
    c.plan(ints([20, 30]))
    x = torch.randn(64, 1, 64, generator=gen(3)).to(DEV)
    c.append(0, x, x + 1)
    c.plan(ints([-3, 0]))
    k, v = c.read(0, 0, 60, torch.float32)
    # int8 codes of one scale a page: half a step of max / 127, twice where the scale grew
    step = float((x.abs().max() + 1) / 127)
    assert (k[:17] - x[:17]).abs().max() <= step and (v[:17] - x[:17] - 1).abs().max() <= step
    assert (k[17:] == 0).all() and (v[17:] == 0).all()
