"""The definitions of the ragged-batch operators (oracle/ragged.py) against
independent ones."""
import numpy as np
import pytest
import torch

from oracle import ragged as og


def test_codes_against_torch():
    b = np.arange(256, dtype=np.uint8)
    t = torch.from_numpy(b).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(og.e4m3_values(), t)
    g = torch.Generator()
    g.manual_seed(0)
    x = torch.cat([torch.randn(20000, generator=g) * s for s in (1e-3, 0.02, 1.0, 100.0)]).clamp(-448, 448)
    mid = torch.from_numpy(t[np.isfinite(t)]).float().sort().values
    x = torch.cat([x, mid, (mid[1:] + mid[:-1]) / 2])           # every code and every tie
    want = x.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(og.encode(x.double().numpy(), "e4m3"), want)
    np.testing.assert_array_equal(og.decode(og.encode(np.array([-200.0, -0.5, 0.5, 1.5, 126.6]), "int8"), "int8"),
                                  [-127, 0, 0, 2, 127])


@pytest.mark.parametrize("hd", [64, 128])
def test_places_are_a_bijection(hd):
    k, v = og._places(hd)
    assert sorted(np.concatenate([k.ravel(), v.ravel()])) == list(range(2 * 16 * hd))
    assert k[3, hd - 1] == og.k_place(3, hd - 1, hd) and v[13, 6] == og.v_place(13, 6, hd)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_append_then_read_is_near(kind):
    rng = np.random.default_rng(0)
    H, hd, n = 2, 64, 40
    pool = np.full((4, H, og.block_bytes(hd)), 0xEE, np.uint8)
    k, v = (rng.standard_normal((n, H, hd)).astype(np.float32) for _ in range(2))
    for i in range(n):                                          # one token a call: scales grow
        og.append(pool, k[i:i + 1], v[i:i + 1], [16 + i], kind)
    rk, rv = og.read(pool, np.arange(16, 16 + n), kind, hd)
    # each growth of the scale re-rounds a code: at most 16 half steps
    for got, x in ((rk, k), (rv, v)):
        top = np.abs(x).max()
        step = top / 127 if kind == "int8" else np.maximum(np.abs(x) * 2.0 ** -3, top / 448 * 2.0 ** -9)
        assert (np.abs(got - x) <= 8 * step).all()
    whole = np.full_like(pool, 0x11)
    og.append(whole, k, v, np.arange(16, 16 + n), kind)         # one call: half a step
    rk, _ = og.read(whole, np.arange(16, 16 + n), kind, hd)
    step = np.abs(k).max() / 127 if kind == "int8" else np.abs(k) * 2.0 ** -3 + np.abs(k).max() / 448 * 2.0 ** -9
    assert (np.abs(rk - k) <= 0.51 * step).all()


def test_attention_against_sdpa():
    rng = np.random.default_rng(1)
    H, G, hd, n = 2, 3, 64, 37
    pool = np.zeros((5, H, og.block_bytes(hd)), np.uint8)
    k, v = (rng.standard_normal((n, H, hd)).astype(np.float32) for _ in range(2))
    slots = [[3, 0, 4][t // 16] * 16 + t % 16 for t in range(n)]
    og.append(pool, k, v, slots, "int8")
    rk, rv = og.read(pool, slots, "int8", hd)
    q = rng.standard_normal((4, H * G, hd))
    table = np.array([[3, 0, 4, -1]], np.int32)
    got = og.attention(q, pool, [n], table, "int8", hd, q_start=[0, 4], max_q=4, window=20)
    pos, at = torch.arange(n), torch.arange(n - 4, n)[:, None]
    mask = (pos <= at) & (pos > at - 20)
    tq = torch.from_numpy(q).transpose(0, 1)
    tk, tv = (torch.from_numpy(x).transpose(0, 1).repeat_interleave(G, 0) for x in (rk, rv))
    want = torch.nn.functional.scaled_dot_product_attention(tq, tk, tv, attn_mask=mask).transpose(0, 1).numpy()
    np.testing.assert_allclose(got, want, atol=1e-12)


def test_plan_keeps_every_page_once():
    rng = np.random.default_rng(2)
    B, max_blocks, n_pages = 6, 5, 22
    lens, table = np.zeros(B, int), np.zeros((B, max_blocks), np.int32)
    free, n_free = np.arange(n_pages, dtype=np.int32), n_pages
    for _ in range(200):
        delta = rng.choice([1, 7, 16, 40, -3, -50, 0], B)
        w = og.block_tables(lens, delta, table, free, n_free, 64)
        lens, table, free, n_free = w["lens"], w["table"], w["free_list"], w["n_free"]
        held = [int(p) for b in range(B) for p in table[b, :og.pages_of(lens[b])]]
        assert sorted(held + [int(p) for p in free[:n_free]]) == list(range(n_pages))
        live = w["slots"][:w["q_start"][-1]]
        assert len(set(live.tolist())) == len(live) and (w["slots"][len(live):] == -1).all()
