"""The ragged-batch operators on the GPU where numbers end: values that are
not finite, weights and scales far apart, limits of lists and tables."""
import numpy as np
import pytest
import torch

import activation_kv_sparsity_b200 as bc
from oracle import ragged as og
from ragged_util import attention_tol, gen, make_pool, to

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
CODES = ["e4m3", "int8"]
DTYPES = [torch.float32, torch.bfloat16]


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def attend(q, pool, lens, table, code, q_start=None, max_q=1, **kw):
    """One call on host data: float64 [n_q][Hq][hd]."""
    P, H, block = pool.shape
    out = torch.full(q.shape, -77.0, dtype=q.dtype, device=DEV)
    scratch = torch.zeros(bc.bc_kv8_attention_scratch_bytes(len(lens), H, q.shape[1] // H, max_q, q.shape[2]),
                          dtype=torch.uint8, device=DEV)
    bc.kv8_attention(q.to(DEV), to(DEV, pool), ints(lens), ints(table), out, scratch, code,
                     q_start=None if q_start is None else ints(q_start), max_q=max_q, **kw)
    assert bc.bc_kv8_attention_status(scratch.data_ptr(), None) == bc.BC_OK
    return out.float().cpu().double().numpy()


# ------------------------------------------------------------------ not finite
def codes_of(pool, page, h, part, hd):
    return pool[page, h][og._places(hd)[part]]


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hd", [64, 128])
def test_append_of_a_value_that_is_not_finite_leaves_zeros(code, dtype, hd):
    """The scale says it; a code that is not a number would reach rows that
    mask the token."""
    H = 2
    pool = make_pool(3, H, hd, code, seed=1)
    k = torch.randn(4, H, hd, generator=gen(2))
    v = torch.randn(4, H, hd, generator=gen(3))
    k[1, 1, 5], v[0, 0, 3], v[3, 1, hd - 1] = float("inf"), float("nan"), float("-inf")
    k, v = k.to(dtype), v.to(dtype)
    dev = to(DEV, pool)
    # a fresh page, then a used one
    for slots in ([16, 17, 18, 19], [2 * 16 + 5 + i for i in range(4)]):
        og.append(pool, k.float().numpy(), v.float().numpy(), slots, code)
        bc.kv8_append(k.to(DEV), v.to(DEV), ints(slots), dev, code)
        got = dev.cpu().numpy()
        np.testing.assert_array_equal(got[..., :32 * hd + 8], pool[..., :32 * hd + 8])
        page, off = slots[0] // 16, slots[0] % 16
        for part, h in ((0, 1), (1, 0), (1, 1)):
            assert np.isnan(og.scale_of(got[page, h], part, hd))
            assert (codes_of(got, page, h, part, hd)[off:off + 4] == 0).all()
    # a finite token behind them: the scale stays, the code is 0
    more = torch.full((1, H, hd), -3.0, dtype=dtype)
    og.append(pool, more.float().numpy(), more.float().numpy(), [20], code)
    bc.kv8_append(more.to(DEV), more.to(DEV), ints([20]), dev, code)
    got = dev.cpu().numpy()
    np.testing.assert_array_equal(got[..., :32 * hd + 8], pool[..., :32 * hd + 8])
    assert (codes_of(got, 1, 0, 1, hd)[4] == 0).all() and (codes_of(got, 1, 0, 0, hd)[4] != 0).all()


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("part", [0, 1])
def test_a_token_that_is_not_finite_stays_with_the_rows_that_see_its_block(code, dtype, hd, part):
    """Drafts over the border of two pages: an infinity in the last token
    reaches no earlier row of the page before; one that only the first row's
    window holds reaches no later row."""
    H, G, n, Q = 1, 2, 33, 8                              # queries at 25 .. 32
    q = torch.randn(Q, H * G, hd, generator=gen(5)).to(dtype)
    for bad, window in ((32, 0), (15, 11), (15, 12)):
        kv = [torch.randn(n, H, hd, generator=gen(6 + i)).to(dtype) for i in range(2)]
        kv[part][bad, 0, 7] = float("inf")
        pool = np.zeros((3, H, og.block_bytes(hd)), np.uint8)
        dev = to(DEV, pool)
        for lo, hi in ((0, 32), (32, 33)):
            bc.kv8_append(kv[0][lo:hi].to(DEV), kv[1][lo:hi].to(DEV), ints(range(lo, hi)), dev, code)
        pool, table = dev.cpu().numpy(), np.array([[0, 1, 2]])
        want = og.attention(q.float().numpy(), pool, [n], table, code, hd, [0, Q], Q, window=window)
        got = attend(q, pool, [n], table, code, [0, Q], Q, window=window)
        sees = np.array([(p >= bad) and (not window or 16 * (bad // 16) + 15 > p - window) for p in range(n - Q, n)])
        assert sees.any() and not sees.all()
        assert np.isnan(got[sees]).all()
        fine = pool.copy()
        fine[np.isnan(fine[:, :, 32 * hd:32 * hd + 8].copy().view(np.float32)).any(-1)] = 0
        tol = attention_tol(want[~sees], q.double().numpy(), fine, code, hd, n, 0.0, None, dtype == torch.bfloat16)
        assert (np.abs(got - want)[~sees] <= tol).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("odd_scale", [None, 52, 31])
def test_codes_that_are_not_numbers_stay_with_the_rows_that_see_them(dtype, hd, odd_scale):
    """Whatever the bytes of a block are: a row that masks a token gets nothing
    of it, a row that sees a value code that is not a number gets NaN in that
    dim only, and everywhere from such a key or scale."""
    H, G, n, Q = 2, 2, 61, 12                             # queries at 49 .. 60, of all tiles of 8 rows
    q = torch.randn(Q, H * G, hd, generator=gen(15)).to(dtype)
    kp, vp = og._places(hd)
    pages = make_pool(4, H, hd, "e4m3", seed=16)
    # (token, dim): seen by all rows, by the later ones, by the earlier ones in a window of 20, one of a later tile
    spots = {"value": [(3, 1), (52, 2), (52, hd - 1), (33, 5), (60, 63), (31, 40)], "key": [(55, 9)]}
    for part, window in (("value", 0), ("value", 20), ("value", 13), ("key", 0), ("key", 9)):
        pool = pages.copy()
        for i, (t, d) in enumerate(spots[part]):
            h = i % 2
            pool[t // 16, h][(vp if part == "value" else kp)[t % 16, d]] = 0x7F if i % 3 else 0xFF
            if t == odd_scale:
                at = 32 * hd + (4 if part == "value" else 0)
                pool[t // 16, h, at:at + 4] = np.array([np.nan], np.float32).view(np.uint8)
        table = np.array([[0, 1, 2, 3]])
        want = og.attention(q.float().numpy(), pool, [n], table, "e4m3", hd, [0, Q], Q, window=window)
        got = attend(q, pool, [n], table, "e4m3", [0, Q], Q, window=window)
        np.testing.assert_array_equal(np.isnan(got), np.isnan(want), err_msg=f"{part} {window}")
        # (every row sees token 52's page: all of it is NaN if a scale there is)
        assert np.isnan(want).any() and (odd_scale == 52 or not np.isnan(want).all())
        tol = attention_tol(np.nan_to_num(want), q.double().numpy(), pages, "e4m3", hd, n, 0.0, None,
                            dtype == torch.bfloat16)
        ok = ~np.isnan(want)
        assert (np.abs(got - want)[ok] <= np.broadcast_to(tol, want.shape)[ok]).all()


# ------------------------------------------------------------------ far apart
@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("at", [0, 60 * 16 + 5])
def test_many_small_weights_beside_a_large_one(code, dtype, at):
    """One token outweighs each of the others by 2^D and has the value 0, so
    that the output is what the others add up to.

    Relative to the output: the logits (base 2, up to 30) have five f32
    roundings, the exponents of the value scales (up to 40) three of 2^-24 of
    themselves, exponentials and the two-part weight 2^-21; 125 pages are summed
    one after the other, each with an error of 2^-23 of the sum, in numerator
    and denominator.  Besides, a weight has an absolute floor, half the smallest
    f16 number, under a largest one of at least 2^13 (2^7 with bf16 outputs,
    whose weights have one part, 2^-11, and are rounded to 2^-8).

    222 sequences of 8 heads: on 148 SMs each is the work of one warp."""
    B, H, hd, n = 222, 8, 64, 2000
    half = dtype == torch.bfloat16
    g = gen(21)
    k, v = torch.zeros(n, 1, hd), 0.5 + 0.5 * torch.rand(n, 1, hd, generator=g)
    k[at, 0, 0], v[at] = 1.0, 0.0
    n_pages = og.pages_of(n)
    one = np.zeros((n_pages, 1, og.block_bytes(hd)), np.uint8)
    og.append(one, k.numpy(), v.numpy(), np.arange(n), code)
    pool = np.repeat(one, H, axis=1)
    table = np.arange(n_pages)[None].repeat(B, 0)
    q = torch.zeros(1, 1, hd)
    q[0, 0, 0] = 1.0
    for D in (10.0, 17.5, 20.3, 23.7, 26.2, 29.8):
        scale = float(np.float32(D * np.log(2.0)))
        want = og.attention(q.numpy(), one, [n], table[:1], code, hd, scale=scale)
        got = attend(q.to(dtype).expand(B, H, hd).contiguous(), pool, [n] * B, table, code, scale=scale)
        rel = (5 * 30 + 3 * 40) * 2.0 ** -24 + 2.0 ** -21 + 2 * 125 * 2.0 ** -23
        tol = np.abs(want) * (rel + (2.0 ** -8 + 2.0 ** -11 if half else 0.0)) + n * 2.0 ** (-32 if half else -38)
        assert (np.abs(got - want) <= tol).all(), (D, float((np.abs(got - want) / np.abs(want)).max()))


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("n", [64, 3000])
def test_values_at_the_end_of_the_normal_numbers(code, n):
    """Value scales of 2^-126.  Relative to the output: exponents of up to 140
    have three roundings of 2^-24 of themselves, weights and exponentials
    2^-20, the sums (n / 16 + 32) 2^-23; the logits (base 2, up to 10) five
    roundings; and an output rounds to a multiple of 2^-149, twice."""
    H, G, hd = 2, 2, 64
    g = gen(31)
    k = 0.3 * torch.randn(n, H, hd, generator=g)
    v = 1e-37 * (0.5 + 0.5 * torch.rand(n, H, hd, generator=g))
    n_pages = og.pages_of(n)
    pool = np.zeros((n_pages, H, og.block_bytes(hd)), np.uint8)
    og.append(pool, k.numpy(), v.numpy(), np.arange(n), code)
    q = 0.5 * torch.randn(1, H * G, hd, generator=g)
    table = np.arange(n_pages)[None]
    want = og.attention(q.numpy(), pool, [n], table, code, hd)
    got = attend(q, pool, [n], table, code)
    rel = 3 * 140 * 2.0 ** -24 + 2.0 ** -20 + 2 * (n / 16 + 32) * 2.0 ** -23 + 2 * 5 * 10 * 2.0 ** -24
    assert (want > 2.0 ** -126).all()
    assert (np.abs(got - want) <= want * rel + 2.0 ** -148).all(), float((np.abs(got - want) / want).max())


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dtype,top", [(torch.float32, 2.0 ** 15), (torch.float32, 2.0 ** 22),
                                       (torch.bfloat16, 2.0 ** 20)])
@pytest.mark.parametrize("hd", [64, 128])
def test_a_query_channel_that_outweighs_the_others(code, dtype, top, hd):
    """A channel of q far above the others, where the keys are 0: the logits
    come from the others, which the tolerance is taken from."""
    H, G, n = 2, 4, 200
    g = gen(41)
    k, v = torch.randn(n, H, hd, generator=g), torch.randn(n, H, hd, generator=g)
    k[..., 9] = 0.0
    n_pages = og.pages_of(n)
    pool = np.zeros((n_pages, H, og.block_bytes(hd)), np.uint8)
    og.append(pool, k.numpy(), v.numpy(), np.arange(n), code)
    q = torch.randn(1, H * G, hd, generator=g).to(dtype)
    q[..., 9] = top
    table = np.arange(n_pages)[None]
    want = og.attention(q.float().numpy(), pool, [n], table, code, hd)
    got = attend(q, pool, [n], table, code)
    rest = q.double().numpy()
    rest[..., 9] = 0.0
    tol = attention_tol(want, rest, pool, code, hd, n, 0.0, None, dtype == torch.bfloat16)
    assert (np.abs(got - want) <= tol).all(), float(np.abs(got - want).max())


@pytest.mark.parametrize("code", CODES)
def test_long_sums_are_not_biased(code):
    """65536 equal weights of values of one sign, all pages of a head in one
    warp (as above), f32.  Relative to the output: log2 of a value scale
    (2^-8.8) is off by 2^-22 of itself, the exponents (up to 16) have three
    roundings, weights and exponentials 2^-20; and of 4096 additions rounded to
    nearest, each off by 0.29 units of 2^-23 in the root mean square, six
    standard deviations.  (Sums cut off instead would be low by up to 4096
    2^-24, 2.4e-4.)"""
    B, H, hd, P, n_pages = 222, 8, 64, 64, 4096
    g = gen(51)
    v = 0.5 + 0.5 * torch.rand(P * 16, 1, hd, generator=g)
    one = np.zeros((P, 1, og.block_bytes(hd)), np.uint8)
    og.append(one, np.zeros(v.shape, np.float32), v.numpy(), np.arange(P * 16), code)
    want = og.read(one, np.arange(P * 16), code, hd)[1].mean(0)
    got = attend(torch.randn(B, H, hd, generator=g), np.repeat(one, H, axis=1), [16 * n_pages] * B,
                 (np.arange(n_pages) % P)[None].repeat(B, 0), code)
    rel = np.log(2.0) * (9 * 2.0 ** -22 + 3 * 16 * 2.0 ** -24) + 2.0 ** -20 + 6 * 0.29 * 4096 ** 0.5 * 2.0 ** -23
    assert (np.abs(got / want - 1) <= rel).all(), (float(np.abs(got / want - 1).max()), rel)


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("swap", [False, True])
def test_value_scales_that_outweigh_the_logits(code, dtype, swap):
    """A page with logit 0 (base 2) and small values, another with logit -D and
    values that make up for it, however far apart both are.  Relative to the
    output: the logits (up to 140) have five roundings, the exponents (up to
    150) four, log2 of a value scale (up to 115) is off by 2^-22 of itself,
    weights and exponentials 2^-20, the output and its bf16 weights as ever.
    Sequences so many that a warp reads both pages of some."""
    B, hd = 2000, 64
    q = torch.zeros(B, 1, hd, dtype=dtype)
    q[:, 0, 0] = 1.0
    for D, low, high in ((95, -100, 0), (97, -97, 3), (130, -75, 58), (110, -60, 50), (138, -100, 45), (60, -60, 1),
                         (100, -105, 10)):
        k, v = torch.zeros(32, 1, hd), torch.ones(32, 1, hd)
        k[16:, 0, 0] = -1.0
        v[:16] *= 2.0 ** low
        v[16:] *= 2.0 ** high
        pool = np.zeros((2, 1, og.block_bytes(hd)), np.uint8)
        og.append(pool, k.numpy(), v.numpy(), np.arange(32), code)
        pages = [[1, 0] if swap else [0, 1]]
        scale = float(np.float32(D * np.log(2.0)))
        want = og.attention(q[:1].float().numpy(), pool, [32], np.array(pages), code, hd, scale=scale)
        got = attend(q, pool, [32] * B, pages * B, code, scale=scale)
        rel = np.log(2.0) * ((5 * 140 + 4 * 150) * 2.0 ** -24 + 115 * 2.0 ** -22) + 2.0 ** -20
        rel += 2.0 ** -8 + 2.0 ** -11 if dtype == torch.bfloat16 else 2.0 ** -24
        assert (np.abs(got / want - 1) <= rel).all(), (D, low, high, float((got / want).min()))


@pytest.mark.parametrize("cap", [1e-50, -1e-50, 1e-39])
def test_attention_refuses_a_cap_that_is_none_in_32_bits(cap):
    pool, q = to(DEV, make_pool(2, 1, 64, "e4m3", seed=1)), torch.zeros(1, 1, 64, device=DEV)
    out = torch.full_like(q, 7.0)
    scratch = torch.zeros(bc.bc_kv8_attention_scratch_bytes(1, 1, 1, 1, 64), dtype=torch.uint8, device=DEV)
    with pytest.raises(ValueError, match="cap"):
        bc.kv8_attention(q, pool, ints([20]), ints([[0, 1]]), out, scratch, "e4m3", cap=cap)
    assert (out == 7).all()


# ------------------------------------------------------------------ logits
@pytest.mark.parametrize("dtype", DTYPES)
def test_repetition_over_its_range(dtype):
    """Penalties from the smallest normal number to the largest.  x / r as a
    product with the reciprocal: two roundings of 2^-24, a reciprocal that is not
    normal itself (of r above 2^126) to half a step of 2^-149, which is 2^-22 of
    it, one step of a result that is not normal, then the output's."""
    reps = np.array([2.0 ** -126, 1.2e-38, 3e-20, 0.7, 1.3, 5e30, 2.0 ** 126, 1e38, 2e38, 3.4e38, -2e38], np.float32)
    x = np.array([1e-3, 2e-6, 3e-30, 5.0, 3e38, -3.0, -2e-3, 0.0, 2e-38], np.float32)
    B, V = len(reps), len(x)
    lg = torch.from_numpy(np.tile(x, (B, 1))).to(dtype)
    hist = np.tile(np.arange(V), B).astype(np.int32)
    start = (np.arange(B + 1) * V).astype(np.int32)
    a, r = lg.double().numpy(), reps.astype(np.float64)[:, None]
    want = np.where(a > 0, a / r, a * r)
    assert not ((np.abs(want) > 3.35e38) & (np.abs(want) < 3.42e38)).any()       # none at the border of infinity
    out = torch.empty_like(lg, device=DEV)
    bc.logits_adjust(lg.to(DEV), out, hist=to(DEV, hist), hist_start=to(DEV, start), repetition=to(DEV, reps))
    got = out.cpu().double().numpy()
    over = np.abs(want) > 3.4e38
    assert (np.isinf(got) == over).all() and (np.sign(got) == np.sign(want))[over].all()
    half = dtype == torch.bfloat16
    rel = 2 * 2.0 ** -24 + (np.abs(r) > 2.0 ** 126) * 2.0 ** -22 + (2.0 ** -8 if half else 0.0)
    tol = np.abs(want) * rel + 2.0 ** -149 + (2.0 ** -134 if half else 0.0)
    assert (np.abs(got - want) <= tol)[~over].all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hist,bias", [(8192, 0), (8191, 2), (8188, 4), (8187, 4), (8187, 9), (8189, 6), (8193, 2),
                                       (4000, 5000), (4001, 4192), (0, 8192), (0, 8195)])
def test_logits_lists_at_the_limit_of_shared_memory(hist, bias, dtype):
    """8192 entries of a row's lists, the history padded to a multiple of 4 and
    then the biases, lie in shared memory; lists that fill it exactly, and cuts
    through either.  Every bias id comes twice, the first and the last entry
    among them, so that some pairs have one on each side of a cut."""
    V, B, g = 20000, 2, gen(hist + bias)
    x = torch.randn(B, V, generator=g).to(dtype)
    h = torch.randint(0, V, (hist,), generator=g).int()
    h[:hist // 3] = h[hist // 3:hist // 3 * 2]                  # ids of the prompt that come up again
    half_b = torch.randperm(V, generator=g)[:(bias + 1) // 2].int()
    ids = torch.cat([half_b, half_b])[:bias].repeat(B)
    kw = dict(repetition=np.float32([1.3, 0.8]), frequency=np.float32([0.2, -0.1]), presence=np.float32([0.1, 0.4]))
    if hist:
        kw.update(hist=h.repeat(B).numpy(), hist_start=np.arange(B + 1, dtype=np.int32) * hist,
                  prompt_len=np.array([hist // 3, 5], np.int32))
    if bias:
        kw.update(bias_ids=ids.numpy(), bias_vals=torch.randn(B * bias, generator=g).numpy(),
                  bias_start=np.arange(B + 1, dtype=np.int32) * bias)
    want = og.logits_adjust(x.double().numpy(), **kw)
    out = torch.full((B, V), 77.0, dtype=dtype, device=DEV)
    bc.logits_adjust(x.to(DEV), out, **{k: to(DEV, v) for k, v in kw.items()})
    # five f32 roundings of values below 2 |x| + 0.2 c + 0.4 + |bias| < 20, then the output's
    tol = 5 * 2.0 ** -24 * 20 + (np.abs(want) * 2.0 ** -8 if dtype == torch.bfloat16 else 0.0)
    assert (np.abs(out.cpu().double().numpy() - want) <= tol).all()


@pytest.mark.parametrize("code", CODES)
def test_dropped_tokens_keep_their_mark_on_the_scale(code):
    """As the definition has it: tokens taken back leave the page's scale, an
    outlier's or one that is not a number, until its token 0 is written again;
    pages given back and pages before are not touched."""
    H, hd = 1, 64
    cache = bc.RaggedCache(1, 1, 4, H, 1, hd, 4, 64, max_q=4, code=code, device=DEV)
    g = gen(61)
    x = lambda n, f=1.0: f * torch.randn(n, H, hd, generator=g).clamp(-3, 3)
    scale = lambda page: float(og.scale_of(cache.pool[0, page, 0].cpu().numpy(), 1, hd))
    pages = []

    def step(delta, v):
        cache.plan(ints([delta]))
        if v is not None:
            cache.append(0, v.to(DEV), v.to(DEV))
        pages[:] = cache.table[0].cpu().tolist()
    step(20, x(20))
    first, second = scale(pages[0]), scale(pages[1])
    step(4, torch.cat([x(3), x(1, 1000.0)]))               # a draft with an outlier, rejected
    coarse = scale(pages[1])
    assert coarse > 100 * second
    step(-4, None)
    step(2, x(2))
    assert scale(pages[1]) == coarse and scale(pages[0]) == first
    step(3, torch.full((3, H, hd), float("inf")))          # one that is not finite
    step(-3, None)
    q, out = torch.randn(1, 1, hd, generator=g).to(DEV), torch.empty(1, 1, hd, device=DEV)
    step(1, x(1))
    cache.attend(0, q, out)
    assert torch.isnan(out).all() and np.isnan(scale(pages[1]))
    cache.attend(0, q, out, pages=ints([[[0]]]), n_sel=ints([1]))
    assert torch.isfinite(out).all()                       # the page before
    step(-8, None)                                         # 15 tokens: the page is given back
    step(3, x(3))
    cache.attend(0, q, out)
    assert torch.isfinite(out).all() and np.isfinite(scale(pages[1])) and scale(pages[0]) >= first
    cache.status()


# ------------------------------------------------------------------ the plan
@pytest.mark.parametrize("B", [1, 3, 200])
def test_plan_that_is_given_back_more_pages_than_there_are(B):
    """Tables that name pages twice: the list of free pages is cut at n_pages,
    and what is in it comes from the right places."""
    rng = np.random.default_rng(B)
    max_blocks, n_pages, n_free, max_tokens = 12, 7, 2, 40
    table = rng.integers(0, n_pages, (B, max_blocks)).astype(np.int32)
    free = rng.permutation(n_pages).astype(np.int32)
    lens = rng.integers(16 * 9, 16 * max_blocks + 1, B).astype(np.int32)
    delta = np.full(B, -2 ** 31, np.int64)
    if B > 1:
        delta[1], lens[1], delta[2] = 33, 17, -70
    want = og.block_tables(lens, delta, table, free, n_free, max_tokens)
    d = dict(lens=ints(lens), delta=ints(delta), table=ints(table), free_list=ints(free), n_free=ints([n_free]),
             lens_out=ints([-7] * B), n_free_out=ints([-7]), q_start=ints([-7] * (B + 1)),
             slots=ints([-7] * max_tokens), positions=ints([-7] * max_tokens), ticket=ints([0]))
    bc.block_tables(**d)
    for name, got in (("table", d["table"]), ("free_list", d["free_list"]), ("n_free", d["n_free_out"]),
                      ("lens", d["lens_out"]), ("q_start", d["q_start"]), ("slots", d["slots"]),
                      ("positions", d["positions"])):
        np.testing.assert_array_equal(got.cpu().numpy(), np.reshape(want[name], got.shape), err_msg=name)
