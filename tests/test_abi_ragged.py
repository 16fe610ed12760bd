"""Refusals of the ragged-batch entry points: on the host, before any launch."""
import ctypes as C

import pytest
import torch

import activation_kv_sparsity_b200 as bc

P = 256          # a non-null, aligned address that no call may reach


def test_sizes():
    assert bc.bc_kv8_pool_bytes(10, 8, 128) == 10 * 8 * (2 * 16 * 128 + 32)
    for bad in ((0, 8, 128), (10, 0, 128), (10, 8, 96), (2 ** 28, 8, 64), (-1, 1, 64)):
        assert bc.bc_kv8_pool_bytes(*bad) == 0
    assert bc.bc_kv8_attention_scratch_bytes(4, 8, 4, 1, 128) > 0
    for bad in ((0, 8, 4, 1, 128), (2049, 8, 4, 1, 128), (4, 0, 4, 1, 128), (4, 8, 9, 1, 128), (4, 8, 4, 0, 128),
                (4, 8, 4, 17, 128), (4, 8, 4, 1, 80), (4, 8, 4, 2 ** 30, 64)):
        assert bc.bc_kv8_attention_scratch_bytes(*bad) == 0


def plan(**over):
    a = dict(batch=2, max_blocks=4, n_pages=8, max_tokens=5, lens=P, delta=P, table=P, free_list=P, n_free=P,
             lens_out=P, n_free_out=P, q_start=P, slots=P, positions=P, ticket=P)
    a.update(over)
    return bc.bc_block_tables(C.byref(bc.bc_block_tables_args(**a)), None)


@pytest.mark.parametrize("over", [dict(batch=0), dict(batch=2049), dict(max_blocks=0), dict(max_blocks=2 ** 28),
                                  dict(n_pages=0), dict(n_pages=2 ** 28), dict(max_tokens=-1)] +
                         [{k: None} for k in ("lens", "delta", "table", "free_list", "n_free", "lens_out",
                                              "n_free_out", "q_start", "slots", "positions", "ticket")])
def test_plan_refuses(over):
    assert plan(**over) == bc.BC_EINVAL
    assert bc.bc_last_error()


def test_append_and_gather_refuse():
    def app(k=P, v=P, dtype=0, ks=512, vs=512, slots=P, n=4, pool=P, typ=0, pages=8, H=4, hd=128):
        return bc.bc_kv8_append(k, v, dtype, ks, vs, slots, n, pool, typ, pages, H, hd, None)

    def gat(pool=P, typ=0, pages=8, H=4, hd=128, slots=P, n=4, k=P, v=P, dtype=0):
        return bc.bc_kv8_gather(pool, typ, pages, H, hd, slots, n, k, v, dtype, None)

    for over in (dict(k=None), dict(v=None), dict(slots=None), dict(pool=None), dict(pool=264), dict(dtype=2),
                 dict(typ=2), dict(typ=-1), dict(n=-1), dict(pages=0), dict(pages=2 ** 28), dict(H=0), dict(hd=96)):
        assert app(**over) == bc.BC_EINVAL, over
        assert gat(**over) == bc.BC_EINVAL, over
    for over in (dict(ks=511), dict(ks=508), dict(vs=514), dict(k=264), dict(v=260, dtype=1), dict(ks=-512)):
        assert app(**over) == bc.BC_EINVAL, over
    for over in (dict(k=264), dict(v=264)):
        assert gat(**over) == bc.BC_EINVAL, over
    assert app(n=2 ** 31 - 1, H=65535, ks=65535 * 128, vs=65535 * 128) == bc.BC_EINVAL
    # nothing to do: fine whatever the pointers
    assert app(n=0, k=None, v=None, slots=None) == bc.BC_OK
    assert gat(n=0, k=None, v=None, slots=None) == bc.BC_OK


def attn(**over):
    a = dict(q=P, out=P, dtype=0, q_stride=4096, n_q=2, pool=P, type=0, n_pages=8, n_kv_heads=8, group=4,
             head_dim=128, batch=2, max_q=1, max_blocks=4, max_sel=0, lens=P, q_start=None, table=P, pages=None,
             n_sel=None, scale=0.1, cap=0.0, window=0, slopes=None, scratch=P, scratch_bytes=1 << 30)
    a.update(over)
    return bc.bc_kv8_attention(C.byref(bc.bc_kv8_attention_args(**a)), None)


@pytest.mark.parametrize("over", [{k: None} for k in ("q", "out", "pool", "lens", "table", "scratch")] +
                         [dict(dtype=2), dict(type=7), dict(q_stride=4095), dict(q_stride=4088), dict(q_stride=4100),
                          dict(n_q=-1), dict(n_pages=0), dict(n_pages=2 ** 28), dict(n_kv_heads=0), dict(group=0),
                          dict(group=9), dict(head_dim=32), dict(batch=0), dict(batch=2049), dict(max_q=0),
                          dict(max_q=17), dict(max_blocks=0), dict(max_blocks=2 ** 28), dict(pages=P),
                          dict(pages=P, n_sel=P, max_sel=0), dict(q=264), dict(out=264), dict(pool=264),
                          dict(scratch=272), dict(cap=-1.0), dict(cap=float("nan")), dict(window=-1),
                          dict(scale=float("nan")), dict(scale=float("inf")),
                          dict(cap=float("inf")), dict(cap=1e-39)])
def test_attention_refuses(over):
    assert attn(**over) == bc.BC_EINVAL
    assert bc.bc_last_error()


def test_attention_refuses_half_a_page_list():
    """Without its lists a count is not taken for "every page"."""
    assert attn(n_sel=P) == bc.BC_EINVAL


def test_attention_small_scratch_and_no_rows():
    need = bc.bc_kv8_attention_scratch_bytes(2, 8, 4, 1, 128)
    assert attn(scratch_bytes=need - 1) == bc.BC_ENOMEM
    assert attn(n_q=0) == bc.BC_OK
    assert bc.bc_kv8_attention(None, None) == bc.BC_EINVAL
    assert bc.bc_kv8_attention_status(None, None) == bc.BC_EINVAL


def logits(**over):
    a = dict(logits=P, out=P, dtype=0, batch=2, vocab=100, stride=100, out_stride=100)
    a.update(over)
    return bc.bc_logits_adjust(C.byref(bc.bc_logits_args(**a)), None)


@pytest.mark.parametrize("over", [dict(logits=None), dict(out=None), dict(dtype=3), dict(batch=0), dict(batch=65536),
                                  dict(vocab=0), dict(stride=99), dict(out_stride=99), dict(vocab=2 ** 31 - 1),
                                  dict(hist=P), dict(hist=P, hist_start=P, n_hist=-1), dict(bias_ids=P),
                                  dict(bias_ids=P, bias_vals=P), dict(bias_ids=P, bias_start=P),
                                  dict(bias_ids=P, bias_vals=P, bias_start=P, n_bias=-1), dict(mask=P, n_masks=1),
                                  dict(logits=258), dict(out=257, dtype=1)])
def test_logits_refuses(over):
    assert logits(**over) == bc.BC_EINVAL
    assert bc.bc_logits_adjust(None, None) == bc.BC_EINVAL


def test_python_wrappers_refuse():
    """Types, shapes and devices that the C interface cannot see."""
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    pool = torch.zeros(2, 1, 32 * 64 + 32, dtype=torch.uint8)
    x = torch.zeros(3, 1, 64)
    with pytest.raises(ValueError, match="pool"):                 # not a CUDA tensor
        bc.kv8_append(x, x, i(3), pool)
    with pytest.raises(ValueError, match="pool"):
        bc.kv8_gather(pool, i(3), x, x)
    with pytest.raises(ValueError, match="pool"):
        bc.kv8_attention(x, pool, i(3), i(3, 2), x, pool)
    with pytest.raises(ValueError, match="CUDA"):
        bc.logits_adjust(torch.zeros(1, 5), torch.zeros(1, 5))
    with pytest.raises(ValueError, match="CUDA"):
        bc.block_tables(i(1), i(1), i(1, 2), i(4), i(1), i(1), i(1), i(2), i(3), i(3), i(1))
    with pytest.raises(ValueError):
        bc.RaggedCache(1, 1, 4, 1, 9, 64, 4, 4, device="cpu")
    with pytest.raises(ValueError, match="code"):
        bc.RaggedCache(1, 1, 4, 1, 4, 64, 4, 4, code="e5m2", device="cpu")
