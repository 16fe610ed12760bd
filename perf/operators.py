"""What is measured of the operators that serve a ragged batch of sequences.

Five operators: the page plan of a batch (block tables, slot map), the append
to and the read-back from an 8-bit paged KV cache (a scale for each page and
kv head, keys and values apart), the attention over that cache, and the
adjustment of logits (penalties, biases, grammar masks).

With ``own`` false, ``run`` computes them in elementary torch operations; with
``own`` true it calls the library's operators.  ``exact`` computes the same
from the definitions in 64 bits.

A block of the cache is one page (16 tokens) of one kv head:
    key codes    [hd / 64][16 tokens][64 dims]
    value codes  [hd / 4][4 token groups][4 dims][4 tokens]
    f32 key scale, f32 value scale, 24 bytes of padding
and the pool is uint8 [n_pages][n_kv_heads][32 hd + 32].
"""
import math

import numpy as np
import torch

own = False

PAGE = 16
DEV = "cuda"
FLT_MIN = 2.0 ** -126
GOLD = 0.6180339887498949


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # a decode step of a small batch: every request takes one token, a few need a page
        dict(name="tables_decode", op="tables", batch=24, max_len=2048, kind="decode"),
        # a scheduling step of a big server: prompts enter, most decode, some leave or take drafts back
        dict(name="tables_mixed", op="tables", batch=1000, max_len=4096, kind="mixed"),
        # a decode step of 256 sequences of the 8B shape: one token each, into half-filled pages
        dict(name="append_decode", op="append", n_seq=256, new=1, heads=8, hd=128, code="e4m3", dtype="bf16"),
        # eight prompts enter the cache, the last page of each partly filled
        dict(name="append_prompt", op="append", n_seq=8, new=3001, heads=8, hd=128, code="int8", dtype="bf16"),
        # the tiny decoder's cache (2 kv heads of 64) read back in fp32
        dict(name="gather_tiny", op="gather", n=333, heads=2, hd=64, code="int8", dtype="f32"),
        # a 32K prefix handed from the 8-bit cache to a bf16 one
        dict(name="gather_prefix", op="gather", n=32768, heads=8, hd=128, code="e4m3", dtype="bf16"),
        # the tiny decoder (8 query heads, 2 kv heads of 64), distance bias, three short sequences
        dict(name="attn_tiny", op="attn", batch=3, max_len=300, heads=2, group=4, hd=64, code="int8",
             dtype="f32", max_q=1, keep=1.0, cap=0.0, window=0, slopes=True),
        # a decode step of 64 sequences of the 8B shape, 1K to 8K tokens each
        dict(name="attn_ragged", op="attn", batch=64, max_len=8192, heads=8, group=4, hd=128, code="e4m3",
             dtype="bf16", max_q=1, keep=1.0, cap=0.0, window=0, slopes=False),
        # drafts of up to four tokens verified, capped scores, a window of 4096 tokens
        dict(name="attn_verify", op="attn", batch=16, max_len=12001, heads=8, group=4, hd=128, code="int8",
             dtype="bf16", max_q=4, keep=1.0, cap=30.0, window=4096, slopes=False),
        # four long sequences, half of the pages selected for each kv head
        dict(name="attn_selected", op="attn", batch=4, max_len=131072, heads=8, group=4, hd=128, code="e4m3",
             dtype="f32", max_q=1, keep=0.5, cap=0.0, window=0, slopes=False),
        # the logits of one sequence, a short history, a few biases
        dict(name="logits_one", op="logits", batch=1, vocab=128256, hist=200, bias=5, masks=0, dtype="f32"),
        # a batch with histories of up to 8K tokens and grammar masks
        dict(name="logits_batch", op="logits", batch=160, vocab=128256, hist=8192, bias=32, masks=16, dtype="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "append", "gather", "attn", "attn", "logits"])
    if op == "tables":
        return dict(op=op, batch=_log(rng, 1, 1024), max_len=_log(rng, 64, 4096),
                    kind=rng.choice(["decode", "mixed"]))
    head = dict(heads=rng.choice([1, 2, 4, 8]), hd=rng.choice([64, 128]), code=rng.choice(["e4m3", "int8"]),
                dtype=rng.choice(["bf16", "f32"]))
    if op == "append":
        n_seq = _log(rng, 1, 256)
        return dict(op=op, n_seq=n_seq, new=rng.choice([1, _log(rng, 1, max(2, 16000 // n_seq))]), **head)
    if op == "gather":
        return dict(op=op, n=_log(rng, 1, 32768), **head)
    if op == "attn":
        max_len = _log(rng, 1, 131072)
        batch = _log(rng, 1, max(1, min(256, 524288 // max_len)))
        group = rng.choice([1, 2, 4, 7, 8])
        long = max_len > 64 and rng.random() < 0.3
        return dict(op=op, batch=batch, max_len=max_len, group=group,
                    max_q=rng.choice([1, 1, 1, rng.randint(2, 8)]) if max_len >= 8 else 1,
                    keep=rng.choice([0.3, 0.5]) if long else 1.0,
                    cap=rng.choice([0.0, 0.0, 30.0]), window=rng.choice([0, 0, _log(rng, 16, 8192)]),
                    slopes=rng.random() < 0.25, **head)
    return dict(op=op, batch=_log(rng, 1, 160), vocab=rng.choice([4096, 32001, 128256]), hist=_log(rng, 1, 8192),
                bias=rng.choice([0, 5, 32]), masks=rng.choice([0, 0, 3, 16]), dtype=rng.choice(["f32", "bf16"]))


# ------------------------------------------------------------------ shapes that follow from a case
def _frac(i):
    return (i * GOLD) % 1.0


def _attn_lens(c):
    """Lengths spread over max_len / 8 .. max_len; the fourth sequence of a batch of five or more is an idle row."""
    lens = [max(1, int(c["max_len"] * 8.0 ** -_frac(i))) for i in range(c["batch"])]
    if len(lens) >= 5:
        lens[3] = 0
    return lens


def _attn_qlens(c):
    return [1 + (i * 5 + c["max_q"] - 1) % c["max_q"] for i in range(c["batch"])]


def _attn_pages(c, n):
    """(first page, pages, kept pages) of a sequence of n tokens."""
    P = -(-n // PAGE)
    return P, (P if c["keep"] >= 1.0 else max(1, math.ceil(c["keep"] * P - 1e-9)))


def _append_off(c):
    """Tokens that each sequence has in its last page already."""
    return [int(16 * _frac(i + 1)) if c["new"] < 64 else (0 if i % 2 == 0 else 9) for i in range(c["n_seq"])]


def _append_new(c):
    return [c["new"] if c["new"] < 4 else max(1, c["new"] - (i * 37) % (c["new"] // 2)) for i in range(c["n_seq"])]


def _tables_requests(c):
    """Lengths and changes of the requests of a planning step."""
    lens, delta = [], []
    for i in range(c["batch"]):
        n = max(1, int(c["max_len"] * 8.0 ** -_frac(i)))
        d = 1
        if c["kind"] == "mixed":
            d = (1, 1, 1, 1, 4, -3, -n, 1)[i % 8]
            if i % 8 == 7:                          # a prompt enters
                n, d = 0, n
        elif i % 6 == 5:                            # an idle row
            n, d = 0, 0
        lens.append(n)
        delta.append(d)
    return lens, delta


def _hist_len(c, i):
    return max(1, int(c["hist"] * 16.0 ** -_frac(i)))


def work(case):
    c = case
    if c["op"] == "tables":
        lens, delta = _tables_requests(c)
        new = sum(d for d in delta if d > 0)
        need = sum(-(-(n + d) // PAGE) - -(-n // PAGE) for n, d in zip(lens, delta) if d > 0)
        back = sum(-(-n // PAGE) - -(-max(0, n + d) // PAGE) for n, d in zip(lens, delta) if d < 0)
        return dict(bytes=4 * (4 * c["batch"] + 2 * new + 2 * need + 2 * back), flops=0)
    size = 4 if c.get("dtype") == "f32" else 2
    if c["op"] == "append":
        new, off = _append_new(c), _append_off(c)
        pages = sum(-(-(o + n) // PAGE) for o, n in zip(off, new))
        old = sum(off)
        e = c["heads"] * c["hd"] * 2
        # new values read and their codes written; every value of the touched pages read back
        total = sum(new) * e * (size + 1) + (sum(new) + old) * e * (1 + size) + pages * c["heads"] * 16 + 4 * sum(new)
        return dict(bytes=total, flops=4 * sum(new) * e)
    if c["op"] == "gather":
        e = c["heads"] * c["hd"] * 2
        return dict(bytes=c["n"] * (e * (1 + size) + 4) + -(-c["n"] // PAGE) * c["heads"] * 8, flops=c["n"] * e)
    if c["op"] == "attn":
        toks, pairs, rows, pages = 0, 0, 0, 0
        for n, ql in zip(_attn_lens(c), _attn_qlens(c)):
            P, K = _attn_pages(c, n)
            span = n if not c["window"] else min(n, c["window"] + ql - 1)
            t = span if c["keep"] >= 1.0 else int(span * K / max(P, 1))
            toks += t
            pages += -(-t // PAGE)
            pairs += t * ql
            rows += ql
        hq = c["heads"] * c["group"]
        return dict(bytes=toks * c["heads"] * c["hd"] * 2 + pages * c["heads"] * 8 + 2 * rows * hq * c["hd"] * size
                    + 4 * pages * (c["heads"] if c["keep"] < 1.0 else 1),
                    flops=4 * pairs * hq * c["hd"])
    hist = sum(_hist_len(c, i) for i in range(c["batch"]))
    mask = c["batch"] * -(-c["vocab"] // 32) * 4 if c["masks"] else 0
    return dict(bytes=2 * c["batch"] * c["vocab"] * size + 4 * hist + 8 * c["batch"] * c["bias"] + mask,
                flops=4 * hist)


# ------------------------------------------------------------------ inputs
def _dtype(c):
    return torch.float32 if c["dtype"] == "f32" else torch.bfloat16


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _int(values):
    return torch.tensor(list(values), dtype=torch.int32, device=DEV)


def _qmax(code):
    return 448.0 if code == "e4m3" else 127.0


def _encode(x, code):
    """Codes of values already divided by their scale."""
    q = _qmax(code)
    x = x.clamp(-q, q)
    if code == "e4m3":
        return x.to(torch.float8_e4m3fn).view(torch.uint8)
    return torch.round(x).to(torch.int8).view(torch.uint8)


def _decode(b, code):
    return b.view(torch.float8_e4m3fn).float() if code == "e4m3" else b.view(torch.int8).float()


def _pack_k(codes):
    """[..., 16, hd] -> [..., 16 hd] in the block's key order."""
    s = codes.shape
    return codes.reshape(*s[:-2], 16, s[-1] // 64, 64).transpose(-3, -2).reshape(*s[:-2], 16 * s[-1])


def _unpack_k(b, hd):
    s = b.shape[:-1]
    return b.reshape(*s, hd // 64, 16, 64).transpose(-3, -2).reshape(*s, 16, hd)


def _pack_v(codes):
    """[..., 16, hd] -> [..., 16 hd] in the block's value order."""
    s = codes.shape
    n = len(s) - 2
    x = codes.reshape(*s[:-2], 4, 4, s[-1] // 4, 4)             # tg, tj, d4, dj
    return x.permute(*range(n), n + 2, n, n + 3, n + 1).reshape(*s[:-2], 16 * s[-1])


def _unpack_v(b, hd):
    s = b.shape[:-1]
    n = len(s)
    x = b.reshape(*s, hd // 4, 4, 4, 4)                         # d4, tg, dj, tj
    return x.permute(*range(n), n + 1, n + 3, n, n + 2).reshape(*s, 16, hd)


def _random_pool(c, n_pages, g):
    """A pool whose pages hold keys N(0, 1) with four channels x 8 and values N(0, 1)."""
    H, hd, code = c["heads"], c["hd"], c["code"]
    pool = torch.zeros(n_pages, H, 32 * hd + 32, dtype=torch.uint8, device=DEV)
    amp = torch.ones(hd, device=DEV)
    amp[[7, hd // 4 + 7, hd // 2 + 6, hd - 5]] = 8.0
    step = max(1, (1 << 25) // (H * 16 * hd))
    for p in range(0, n_pages, step):
        n = min(step, n_pages - p)
        scales = []
        for part, mul, pack in ((0, amp, _pack_k), (1, None, _pack_v)):
            x = torch.randn(n, H, 16, hd, generator=g, device=DEV)
            if mul is not None:
                x *= mul
            s = x.abs().amax(dim=(2, 3)) / _qmax(code)
            pool[p:p + n, :, part * 16 * hd:(part + 1) * 16 * hd] = pack(_encode(x / s[..., None, None], code))
            scales.append(s)
        pool[p:p + n, :, 32 * hd:32 * hd + 8] = torch.stack(scales, -1).contiguous().view(torch.uint8)
    return pool


def _slots_of(pages, first, count):
    """Slots of tokens first .. first + count - 1 of a sequence with these pages."""
    pos = torch.arange(first, first + count, device=DEV)
    return (pages[pos // PAGE].long() * PAGE + pos % PAGE).int()


def prepare(case, seed):
    c = case
    g = _gen(seed)
    if c["op"] == "tables":
        lens, delta = _tables_requests(c)
        B = c["batch"]
        max_blocks = -(-max(max(n + d for n, d in zip(lens, delta)), max(lens), 1) // PAGE) + 1
        held = [-(-n // PAGE) for n in lens]
        need = sum(max(0, -(-(n + d) // PAGE) - h) for n, d, h in zip(lens, delta, held))
        n_pages = sum(held) + need + 7
        perm = torch.randperm(n_pages, generator=g, device=DEV).int()
        table = torch.full((B, max_blocks), -1, dtype=torch.int32, device=DEV)
        at = 0
        for b in range(B):
            table[b, :held[b]] = perm[at:at + held[b]]
            at += held[b]
        free = torch.full((n_pages,), -1, dtype=torch.int32, device=DEV)
        free[:n_pages - at] = perm[at:]
        max_tokens = sum(d for d in delta if d > 0) + 5
        e = lambda *s: torch.empty(*s, dtype=torch.int32, device=DEV)
        return dict(case=c, lens=_int(lens), delta=_int(delta), table=table, free=free, n_free=_int([n_pages - at]),
                    lens_out=e(B), n_free_out=e(1), q_start=e(B + 1), slots=e(max_tokens), positions=e(max_tokens),
                    ticket=torch.zeros(1, dtype=torch.int32, device=DEV))
    if c["op"] == "append":
        H, hd = c["heads"], c["hd"]
        new, off = _append_new(c), _append_off(c)
        n = sum(new)
        pages = [-(-(o + m) // PAGE) for o, m in zip(off, new)]
        n_pages = sum(pages) + 3
        perm = torch.randperm(n_pages, generator=g, device=DEV).int()
        slots, read, at = [], [], 0
        for o, m, p in zip(off, new, pages):
            mine = perm[at:at + p]
            at += p
            slots.append(_slots_of(mine, o, m))
            read.append(_slots_of(mine, 0, o + m))
        slots, read = torch.cat(slots), torch.cat(read)
        qkv = torch.randn(n, (4 * H + 2 * H) * hd, generator=g, device=DEV)      # the fused projection's rows
        qkv[:, 4 * H * hd:5 * H * hd].view(n, H, hd)[..., 7] *= 8.0
        qkv = qkv.to(_dtype(c))
        k = qkv[:, 4 * H * hd:5 * H * hd].view(n, H, hd)
        v = qkv[:, 5 * H * hd:].view(n, H, hd)
        kr = torch.empty(read.numel(), H, hd, dtype=_dtype(c), device=DEV)
        return dict(case=c, pool=_random_pool(c, n_pages, g), k=k, v=v, slots=slots, read=read, k_out=kr,
                    v_out=torch.empty_like(kr))
    if c["op"] == "gather":
        P = -(-c["n"] // PAGE)
        pool = _random_pool(c, P + 2, g)
        pages = torch.randperm(P + 2, generator=g, device=DEV).int()[:P]
        slots = _slots_of(pages, 0, c["n"])
        k = torch.empty(c["n"], c["heads"], c["hd"], dtype=_dtype(c), device=DEV)
        return dict(case=c, pool=pool, slots=slots, k_out=k, v_out=torch.empty_like(k))
    if c["op"] == "attn":
        lens, ql = _attn_lens(c), _attn_qlens(c)
        B, H, G, hd = c["batch"], c["heads"], c["group"], c["hd"]
        blocks = [-(-n // PAGE) for n in lens]
        n_pages = sum(blocks) + 1
        perm = torch.randperm(n_pages, generator=g, device=DEV).int()
        table = torch.full((B, max(max(blocks), 1) + 1), -1, dtype=torch.int32, device=DEV)
        at = 0
        for b in range(B):
            table[b, :blocks[b]] = perm[at:at + blocks[b]]
            at += blocks[b]
        pages = n_sel = None
        kept = [_attn_pages(c, n)[1] if n else 0 for n in lens]
        if c["keep"] < 1.0:
            pages = torch.zeros(B, H, max(kept), dtype=torch.int32, device=DEV)
            for b in range(B):
                P = blocks[b]
                if not P:
                    continue
                score = torch.rand(H, P, generator=g, device=DEV)
                score[:, 0] = score[:, -1] = 2.0                  # the first and the last page are always kept
                pages[b, :, :kept[b]] = score.topk(kept[b], dim=1).indices.sort(dim=1).values.int()
            n_sel = _int(kept)
        starts = [0]
        for x in ql:
            starts.append(starts[-1] + x)
        q = torch.randn(starts[-1], H * G, hd, generator=g, device=DEV).to(_dtype(c))
        slopes = None
        if c["slopes"]:
            slopes = torch.tensor([2.0 ** (-8.0 * (i + 1) / (H * G)) for i in range(H * G)], device=DEV)
        # 16 MB of scratch serve every size here
        return dict(case=c, pool=_random_pool(c, n_pages, g), q=q, out=torch.empty_like(q), lens=_int(lens),
                    q_start=_int(starts) if c["max_q"] > 1 else None, starts=starts, lens_host=lens, table=table,
                    pages=pages, n_sel=n_sel, kept=kept, slopes=slopes,
                    scratch=torch.zeros(16 << 20, dtype=torch.uint8, device=DEV))
    B, V = c["batch"], c["vocab"]
    logits = (2.0 * torch.randn(B, V, generator=g, device=DEV)).to(_dtype(c))
    hl = [_hist_len(c, i) for i in range(B)]
    hs = [0]
    for n in hl:
        hs.append(hs[-1] + n)
    # token ids of text: few frequent ones, many rare ones
    u = torch.rand(hs[-1], generator=g, device=DEV)
    hist = (V ** u - 1.0).int().clamp(0, V - 1)
    state = dict(case=c, logits=logits, out=torch.empty_like(logits), hist=hist, hist_start=_int(hs),
                 prompt_len=_int(n // 2 for n in hl),
                 repetition=1.0 + 0.3 * torch.rand(B, generator=g, device=DEV),
                 frequency=0.5 * torch.rand(B, generator=g, device=DEV),
                 presence=0.5 * torch.rand(B, generator=g, device=DEV),
                 bias_ids=None, bias_vals=None, bias_start=None, mask=None, mask_row=None)
    if c["bias"]:
        state["bias_ids"] = torch.randint(0, V, (B * c["bias"],), generator=g, device=DEV).int()
        state["bias_vals"] = 4.0 * torch.randn(B * c["bias"], generator=g, device=DEV)
        state["bias_start"] = _int(range(0, B * c["bias"] + 1, c["bias"]))
    if c["masks"]:
        W = -(-V // 32)
        state["mask"] = torch.randint(-2 ** 31, 2 ** 31, (c["masks"], W), generator=g, device=DEV).int()
        state["mask_row"] = _int((i % (c["masks"] + 1)) - 1 for i in range(B))     # -1: no mask
    return state


# ------------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


def _own_tables(s):
    import activation_kv_sparsity_b200 as bc
    bc.block_tables(s["lens"], s["delta"], s["table"], s["free"], s["n_free"], s["lens_out"], s["n_free_out"],
                    s["q_start"], s["slots"], s["positions"], s["ticket"])
    return [s[k] for k in ("table", "free", "lens_out", "n_free_out", "q_start", "slots", "positions")]


def _own_append(s):
    import activation_kv_sparsity_b200 as bc
    code = s["case"]["code"]
    bc.kv8_append(s["k"], s["v"], s["slots"], s["pool"], code)
    bc.kv8_gather(s["pool"], s["read"], s["k_out"], s["v_out"], code)
    return [s["k_out"], s["v_out"]]


def _own_gather(s):
    import activation_kv_sparsity_b200 as bc
    bc.kv8_gather(s["pool"], s["slots"], s["k_out"], s["v_out"], s["case"]["code"])
    return [s["k_out"], s["v_out"]]


def _own_attn(s):
    import activation_kv_sparsity_b200 as bc
    c = s["case"]
    bc.kv8_attention(s["q"], s["pool"], s["lens"], s["table"], s["out"], s["scratch"], c["code"],
                     q_start=s["q_start"], max_q=c["max_q"], pages=s["pages"], n_sel=s["n_sel"], cap=c["cap"],
                     window=c["window"], slopes=s["slopes"])
    return s["out"]


def _own_logits(s):
    import activation_kv_sparsity_b200 as bc
    bc.logits_adjust(s["logits"], s["out"], hist=s["hist"], hist_start=s["hist_start"], prompt_len=s["prompt_len"],
                     repetition=s["repetition"], frequency=s["frequency"], presence=s["presence"],
                     bias_ids=s["bias_ids"], bias_vals=s["bias_vals"], bias_start=s["bias_start"], mask=s["mask"],
                     mask_row=s["mask_row"])
    return s["out"]


_OWN = dict(tables=_own_tables, append=_own_append, gather=_own_gather, attn=_own_attn, logits=_own_logits)


def _excl(x):
    return torch.cumsum(x, 0) - x


def _plain_tables(s):
    lens, delta, table, free = s["lens"].long(), s["delta"].long(), s["table"], s["free"]
    B, max_blocks = table.shape
    max_tokens, n_pages = s["slots"].numel(), free.numel()
    n_free = s["n_free"].long()[0]
    zero = torch.zeros_like(lens)
    ceil = lambda x: (x + PAGE - 1) // PAGE
    held = ceil(lens)
    back = torch.where(delta < 0, held - ceil((lens + delta).clamp(min=0)), zero)
    back_at = _excl(back)
    n_back = back.sum()
    cand = torch.where((delta > 0) & (lens + delta <= max_blocks * PAGE), delta, zero)
    cand = torch.where(_excl(cand) + cand <= max_tokens, cand, zero)
    need = ceil(lens + cand) - held
    need = torch.where(cand > 0, need, zero)
    need_at = _excl(need)
    ok = (need == 0) | (need_at + need <= n_free + n_back)
    grant = torch.where(ok, cand, zero)
    take = torch.where(ok, need, zero)
    n_take = take.sum()
    start = torch.cat([zero[:1], torch.cumsum(grant, 0)])
    # the pool of free pages: the free list, then the pages given back
    back_end = back_at + back
    r = torch.arange(n_pages, device=DEV)
    rb = torch.searchsorted(back_end, r, right=True).clamp(max=B - 1)
    kept = held - back
    ro = (kept[rb] + r - back_at[rb]).clamp(0, max_blocks - 1)
    given = table[rb, ro]                                         # r-th page given back
    idx = torch.arange(n_pages, device=DEV)
    combined = torch.where(idx < n_free, free, given[(idx - n_free).clamp(0, n_pages - 1)])
    left = n_free + n_back - n_take
    # pages taken: the top of the list first
    j = torch.arange(n_pages, device=DEV)
    take_end = need_at + take
    page_j = combined[(n_free + n_back - 1 - j).clamp(0, n_pages - 1)]
    blk = torch.arange(max_blocks, device=DEV)[None, :]
    is_new = (blk >= held[:, None]) & (blk < (held + take)[:, None])
    jj = (need_at[:, None] + blk - held[:, None]).clamp(0, n_pages - 1)
    new_table = torch.where(is_new, page_j[jj], table)
    new_free = torch.where((idx >= n_free) & (idx < left), combined, free)
    t = torch.arange(max_tokens, device=DEV)
    tb = torch.searchsorted(start[1:], t, right=True).clamp(max=B - 1)
    pos = lens[tb] + t - start[tb]
    page = new_table[tb, (pos // PAGE).clamp(0, max_blocks - 1)].long()
    live = t < start[B]
    minus = torch.full_like(t, -1)
    slots = torch.where(live, page * PAGE + pos % PAGE, minus)
    positions = torch.where(live, pos, minus)
    lens_out = torch.where(delta < 0, (lens + delta).clamp(min=0), lens + grant)
    table.copy_(new_table)
    free.copy_(new_free)
    return [table, free, lens_out.int(), left.reshape(1).int(), start.int(), slots.int(), positions.int()]


def _plain_write(pool, x, slots, part, c):
    """Writes the rows x [n][H][hd] into the pool's keys (part 0) or values (1)."""
    H, hd, code = c["heads"], c["hd"], c["code"]
    n_pages = pool.shape[0]
    x = x.float()
    page, off = slots.long() // PAGE, slots.long() % PAGE
    amax = torch.zeros(n_pages, H, device=DEV)
    amax.scatter_reduce_(0, page[:, None].expand(-1, H), x.abs().amax(-1), "amax")
    first = torch.full((n_pages,), PAGE, dtype=torch.long, device=DEV)
    first.scatter_reduce_(0, page, off, "amin")
    sc = pool[:, :, 32 * hd + 4 * part:32 * hd + 4 * part + 4].contiguous().view(torch.float32)[..., 0]
    touched = first < PAGE
    s_new = torch.where(amax > 0, (amax / _qmax(code)).clamp(min=FLT_MIN), torch.zeros_like(amax))
    s_old = torch.where((first > 0)[:, None], sc, torch.zeros_like(sc))
    s = torch.maximum(s_old, s_new)
    inv = torch.where(s > 0, 1.0 / s, torch.zeros_like(s))
    codes = pool[:, :, part * 16 * hd:(part + 1) * 16 * hd]
    codes = _unpack_k(codes, hd) if part == 0 else _unpack_v(codes, hd)      # [pages, H, 16, hd]
    old = _encode(_decode(codes.contiguous(), code) * s_old[..., None, None] * inv[..., None, None], code)
    tok = torch.arange(PAGE, device=DEV)
    was = tok[None] < first[:, None]
    new = torch.where((was & touched[:, None])[:, None, :, None], old, codes)
    new = torch.where(((first == 0)[:, None] & ~was)[:, None, :, None], torch.zeros_like(new), new)
    new[page, :, off] = _encode(x * inv[page][..., None], code)
    pool[:, :, part * 16 * hd:(part + 1) * 16 * hd] = torch.where(
        touched[:, None, None], _pack_k(new) if part == 0 else _pack_v(new),
        pool[:, :, part * 16 * hd:(part + 1) * 16 * hd])
    s = torch.where(touched[:, None], s, sc)
    pool[:, :, 32 * hd + 4 * part:32 * hd + 4 * part + 4] = s[..., None].contiguous().view(torch.uint8)


def _plain_read(pool, slots, c):
    hd, code = c["hd"], c["code"]
    page, off = slots.long() // PAGE, slots.long() % PAGE
    sc = pool[:, :, 32 * hd:32 * hd + 8].contiguous().view(torch.float32)    # [pages, H, 2]
    out = []
    for part, unpack in ((0, _unpack_k), (1, _unpack_v)):
        codes = unpack(pool[:, :, part * 16 * hd:(part + 1) * 16 * hd], hd)
        x = _decode(codes[page, :, off].contiguous(), code)
        out.append((x * sc[page][:, :, part, None]).to(_dtype(c)))
    return out


def _plain_append(s):
    c = s["case"]
    _plain_write(s["pool"], s["k"], s["slots"], 0, c)
    _plain_write(s["pool"], s["v"], s["slots"], 1, c)
    return _plain_read(s["pool"], s["read"], c)


def _plain_gather(s):
    return _plain_read(s["pool"], s["slots"], s["case"])


def _plain_attn(s):
    """All sequences at once, padded to the longest."""
    c = s["case"]
    H, G, hd, code, B, Q = c["heads"], c["group"], c["hd"], c["code"], c["batch"], c["max_q"]
    q, lens = s["q"], s["lens"].long()
    start = torch.arange(B + 1, device=DEV) if s["q_start"] is None else s["q_start"].long()
    n_q = start[1:] - start[:-1]
    if s["pages"] is None:
        logical = torch.arange(s["table"].shape[1], device=DEV).expand(B, 1, -1)
        live = logical * PAGE < lens[:, None, None]
    else:
        logical = s["pages"].long()                                          # [B, H, K]
        live = (torch.arange(logical.shape[2], device=DEV) < s["n_sel"][:, None]).unsqueeze(1).expand(logical.shape)
    live = live & (logical < s["table"].shape[1])
    page = s["table"].long().gather(1, torch.where(live, logical, torch.zeros_like(logical)).flatten(1)).view(logical.shape)
    page = torch.where(live, page, torch.zeros_like(page))
    blk = s["pool"][page, torch.arange(H, device=DEV)[:, None]]              # [B, H, K, block bytes]
    sc = blk[..., 32 * hd:32 * hd + 8].contiguous().view(torch.float32)
    k = (_decode(_unpack_k(blk[..., :16 * hd], hd), code) * sc[..., 0, None, None]).reshape(B, H, -1, hd)
    v = (_decode(_unpack_v(blk[..., 16 * hd:32 * hd], hd), code) * sc[..., 1, None, None]).reshape(B, H, -1, hd)
    pos = (logical[..., None] * PAGE + torch.arange(PAGE, device=DEV)).flatten(2)[:, :, None, None]
    row = (start[:-1, None] + torch.arange(Q, device=DEV)).clamp(max=q.shape[0] - 1)         # [B, Q]
    qq = q[row].float().view(B, Q, H, G, hd).permute(0, 2, 3, 1, 4)          # [B, H, G, Q, hd]
    qpos = (lens - n_q)[:, None] + torch.arange(Q, device=DEV)
    qpos = qpos.view(B, 1, 1, Q, 1)
    sco = (qq.reshape(B, H, G * Q, hd) @ k.transpose(2, 3)).view(B, H, G, Q, -1) / math.sqrt(hd)
    if c["cap"]:
        sco = c["cap"] * torch.tanh(sco / c["cap"])
    if s["slopes"] is not None:
        sco = sco - s["slopes"].view(H, G, 1, 1) * (qpos - pos)
    keep = live.repeat_interleave(PAGE, -1)[:, :, None, None] & (pos <= qpos)
    if c["window"]:
        keep = keep & (pos > qpos - c["window"])
    sco = torch.where(keep, sco, torch.full((), -math.inf, device=DEV))
    top = sco.amax(-1, keepdim=True)
    p = torch.exp(sco - torch.where(top == -math.inf, torch.zeros_like(top), top))
    tot = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ v).view(B, H, G, Q, hd)
    o = torch.where(tot > 0, o / tot, torch.zeros_like(o)).permute(0, 3, 1, 2, 4).reshape(B, Q, H * G, hd)
    mine = torch.arange(Q, device=DEV) < n_q[:, None]
    out = torch.zeros(q.shape, dtype=torch.float32, device=DEV)
    at = torch.where(mine, row, torch.full_like(row, q.shape[0])).flatten()
    return torch.cat([out, out[:1]]).index_copy_(0, at, o.flatten(0, 1))[:-1].to(q.dtype)


def _plain_logits(s):
    c = s["case"]
    B, V = c["batch"], c["vocab"]
    x = s["logits"].float()
    i = torch.arange(s["hist"].numel(), device=DEV)
    row = torch.searchsorted(s["hist_start"][1:].long(), i, right=True)
    flat = row * V + s["hist"].long()
    is_out = i >= s["hist_start"].long()[row] + s["prompt_len"].long()[row]
    seen = torch.zeros(B * V, device=DEV).index_put_((flat,), torch.ones((), device=DEV)).view(B, V)
    count = torch.zeros(B * V, device=DEV).index_add_(0, flat, is_out.float()).view(B, V)
    rep = s["repetition"][:, None]
    x = torch.where(seen > 0, torch.where(x > 0, x / rep, x * rep), x)
    x = x - (s["frequency"][:, None] * count + s["presence"][:, None] * (count > 0))
    if s["bias_ids"] is not None:
        j = torch.arange(s["bias_ids"].numel(), device=DEV)
        brow = torch.searchsorted(s["bias_start"][1:].long(), j, right=True)
        last = torch.full((B * V,), -1, dtype=torch.long, device=DEV)        # an id twice: the last entry counts
        last.scatter_reduce_(0, brow * V + s["bias_ids"].long(), j, "amax")
        last = last.view(B, V)
        x = torch.where(last >= 0, x + s["bias_vals"][last.clamp(min=0)], x)
    if s["mask"] is not None:
        v = torch.arange(V, device=DEV)
        bit = (s["mask"][s["mask_row"].clamp(min=0).long()][:, v // 32] >> (v % 32)) & 1
        x = torch.where((bit == 1) | (s["mask_row"] < 0)[:, None], x, torch.full_like(x, -math.inf))
    return x.to(s["logits"].dtype)


_PLAIN = dict(tables=_plain_tables, append=_plain_append, gather=_plain_gather, attn=_plain_attn, logits=_plain_logits)


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return _EXACT[case["op"]](s)


def _exact_tables(s):
    """The plan step by step, one request after the other, on the host."""
    h = {k: s[k].cpu().numpy().astype(np.int64) for k in ("lens", "delta", "table", "free", "n_free")}
    table, free, nf = h["table"], h["free"], int(h["n_free"][0])
    B, max_blocks = table.shape
    max_tokens = s["slots"].numel()
    old = table.copy()
    pile = list(free[:nf])
    lens = h["lens"].copy()
    for b in range(B):
        n, d = int(h["lens"][b]), int(h["delta"][b])
        if d < 0:
            m = max(0, n + d)
            pile += [int(p) for p in old[b, -(-m // PAGE):-(-n // PAGE)]]
            lens[b] = m
    slots = np.full(max_tokens, -1, np.int64)
    positions = np.full(max_tokens, -1, np.int64)
    start, used, asked, wanted, room = [0], 0, 0, 0, len(pile)
    for b in range(B):
        n, d = int(h["lens"][b]), int(h["delta"][b])
        ok = d > 0 and n + d <= max_blocks * PAGE
        if ok:
            asked += d
            ok = asked <= max_tokens
        if ok:
            need = -(-(n + d) // PAGE) - -(-n // PAGE)
            wanted += need
            ok = need == 0 or wanted <= room
        if ok:
            for i in range(need):
                table[b, -(-n // PAGE) + i] = pile.pop()
            pos = np.arange(n, n + d)
            slots[used:used + d] = table[b, pos // PAGE] * PAGE + pos % PAGE
            positions[used:used + d] = pos
            used += d
            lens[b] = n + d
        start.append(used)
    if len(pile) > nf:
        free[nf:len(pile)] = pile[nf:]
    out = [table, free, lens, np.array([len(pile)]), np.array(start), slots, positions]
    return [torch.from_numpy(np.ascontiguousarray(x)).to(DEV) for x in out]


def _v_index(hd):
    t, d = np.meshgrid(np.arange(16), np.arange(hd), indexing="ij")
    return torch.from_numpy((d // 4) * 64 + (t // 4) * 16 + (d % 4) * 4 + t % 4).to(DEV)


def _k_index(hd):
    t, d = np.meshgrid(np.arange(16), np.arange(hd), indexing="ij")
    return torch.from_numpy((d // 64) * 1024 + t * 64 + d % 64).to(DEV)


def _values64(blocks, part, c):
    """Values in 64 bits of blocks [..., bytes], by each value's place: [..., 16, hd]."""
    hd = c["hd"]
    at = (_k_index(hd) if part == 0 else 16 * hd + _v_index(hd)).reshape(-1)
    b = blocks.index_select(-1, at).reshape(*blocks.shape[:-1], 16, hd).contiguous()
    x = (b.view(torch.float8_e4m3fn).to(torch.float32) if c["code"] == "e4m3" else b.view(torch.int8)).double()
    lo = 32 * hd + 4 * part
    return x * blocks[..., lo:lo + 4].contiguous().view(torch.float32).double()[..., None]


def _round8(x, code):
    q = _qmax(code)
    x = x.clamp(-q, q)
    if code == "int8":
        return torch.round(x)
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))).clamp(min=-6)
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-q, q)


def _exact_append(s):
    c = s["case"]
    slots, read, code = s["slots"].long(), s["read"].long(), c["code"]
    outs = []
    # token places of the touched pages, in the order of the pages' first appearance
    pages = torch.unique(slots // PAGE)
    where = torch.full((s["pool"].shape[0],), -1, dtype=torch.long, device=DEV)
    where[pages] = torch.arange(pages.numel(), device=DEV)
    for part, x in ((0, s["k"]), (1, s["v"])):
        x = x.double()
        val = _values64(s["pool"][pages], part, c).transpose(1, 2).clone()          # [pages, 16, H, hd]
        new = torch.zeros(val.shape[:2], dtype=torch.bool, device=DEV)
        new[where[slots // PAGE], slots % PAGE] = True
        first = new.int().argmax(1)
        lo = 32 * c["hd"] + 4 * part
        s_old = s["pool"][pages][:, :, lo:lo + 4].contiguous().view(torch.float32)[..., 0].double()
        s_old = torch.where((first > 0)[:, None], s_old, torch.zeros_like(s_old))
        fresh = torch.zeros_like(val)
        fresh[where[slots // PAGE], slots % PAGE] = x
        top = fresh.abs().amax(dim=(1, 3)) / _qmax(code)
        scale = torch.maximum(torch.where(top > 0, top.clamp(min=FLT_MIN), top), s_old)[:, None, :, None]
        val = torch.where(new[..., None, None], fresh, val)
        val = _round8(torch.where(scale > 0, val / scale, torch.zeros_like(val)), code) * scale
        outs.append(val[where[read // PAGE], read % PAGE])
    return outs


def _exact_gather(s):
    c = s["case"]
    slots = s["slots"].long()
    outs = []
    for part in (0, 1):
        res = torch.empty(slots.numel(), c["heads"], c["hd"], dtype=torch.float64, device=DEV)
        for i in range(0, slots.numel(), 4096):
            p = slots[i:i + 4096]
            v = _values64(s["pool"][p // PAGE], part, c)                             # [n, H, 16, hd]
            res[i:i + 4096] = v[torch.arange(p.numel(), device=DEV), :, p % PAGE]
        outs.append(res)
    return outs


def _exact_attn(s):
    c = s["case"]
    H, G, hd = c["heads"], c["group"], c["hd"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    for b in range(c["batch"]):
        n, lo, hi = s["lens_host"][b], s["starts"][b], s["starts"][b + 1]
        if n == 0:
            continue
        for h in range(H):
            logical = torch.arange(-(-n // PAGE), device=DEV) if s["pages"] is None \
                else s["pages"][b, h, :s["kept"][b]].long()
            blk = s["pool"][s["table"][b][logical].long(), h]
            pos = (logical[:, None] * PAGE + torch.arange(PAGE, device=DEV)).reshape(-1)
            ok = pos < n
            k = _values64(blk, 0, c).reshape(-1, hd)[ok]
            v = _values64(blk, 1, c).reshape(-1, hd)[ok]
            pos = pos[ok]
            for i in range(hi - lo):
                at = n - (hi - lo) + i
                see = pos <= at
                if c["window"]:
                    see &= pos > at - c["window"]
                if at < 0 or not bool(see.any()):
                    continue
                x = k[see] @ s["q"][lo + i, h * G:(h + 1) * G].double().T / math.sqrt(hd)      # [tokens, G]
                if c["cap"]:
                    x = c["cap"] * torch.tanh(x / c["cap"])
                if s["slopes"] is not None:
                    x = x + s["slopes"][h * G:(h + 1) * G].double() * (pos[see] - at).double()[:, None]
                out[lo + i, h * G:(h + 1) * G] = torch.softmax(x, 0).T @ v[see]
    return out


def _exact_logits(s):
    c = s["case"]
    V = c["vocab"]
    out = s["logits"].double().clone()
    hs = s["hist_start"].tolist()
    pl = s["prompt_len"].tolist()
    for b in range(c["batch"]):
        h = s["hist"][hs[b]:hs[b + 1]].long()
        seen = torch.unique(h)
        ids, cnt = torch.unique(h[pl[b]:], return_counts=True)
        r, f, p = (float(s[k][b]) for k in ("repetition", "frequency", "presence"))
        x = out[b]
        x[seen] = torch.where(x[seen] > 0, x[seen] / r, x[seen] * r)
        x[ids] -= f * cnt.double() + p
        if s["bias_ids"] is not None:
            lo, hi = s["bias_start"][b:b + 2].tolist()
            add = dict(zip(s["bias_ids"][lo:hi].tolist(), s["bias_vals"][lo:hi].double().tolist()))
            keys = torch.tensor(list(add), device=DEV)
            x[keys] += torch.tensor(list(add.values()), dtype=torch.float64, device=DEV)
        if s["mask"] is not None and int(s["mask_row"][b]) >= 0:
            words = s["mask"][int(s["mask_row"][b])].cpu().numpy().view(np.uint8)
            bits = torch.from_numpy(np.unpackbits(words, bitorder="little")[:V].copy()).to(DEV)
            x[bits == 0] = -math.inf
    return out


_EXACT = dict(tables=_exact_tables, append=_exact_append, gather=_exact_gather, attn=_exact_attn, logits=_exact_logits)
