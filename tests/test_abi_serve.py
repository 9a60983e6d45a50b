"""The operators around the paged cache reject bad arguments before anything reaches the GPU."""
import ctypes

import pytest
import torch

import nucleus_token_sampler_gb300 as tps
from nucleus_token_sampler_gb300 import decode

FAKE = 0x10000  # never dereferenced: every call below fails validation first, or has nothing to do


def prompt(**kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, out=FAKE, cu_seqlens=FAKE, T=10, B=2, q_ld=768, q_hd=64, k_ld=768, k_hd=64, v_ld=768, v_hd=64,
             n_q_heads=8, n_k_heads=2, head_dim=64, scale=0.125)
    a.update(kw)
    return tps.load().tps_prompt_attention(ctypes.byref(decode._Prompt(**a)), None)


@pytest.mark.parametrize("kw,rc", [
    (dict(T=-1), 1), (dict(T=2 ** 31 - 2 ** 16 + 1), 1), (dict(B=-1), 1), (dict(B=2 ** 31), 1), (dict(n_q_heads=0), 1), (dict(n_k_heads=0), 1),
    (dict(n_q_heads=7), 1), (dict(n_q_heads=65536), 1), (dict(head_dim=96), 1), (dict(head_dim=0), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(scale=3e38), 1), (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(out=None), 1), (dict(cu_seqlens=None), 1),
    (dict(q_ld=60), 1), (dict(q_ld=100), 1), (dict(k_hd=0), 1), (dict(v_hd=-64), 1), (dict(v_ld=1 << 40), 1), (dict(q=FAKE + 8), 4),
    (dict(k=FAKE + 2), 4), (dict(v=FAKE + 4), 4), (dict(out=FAKE + 8), 4), (dict(out_lse=FAKE + 2), 4), (dict(cu_seqlens=FAKE + 1), 4),
    (dict(out_status=FAKE + 2), 4), (dict(T=2 ** 31 - 2 ** 16, n_q_heads=2048, n_k_heads=1024, q_ld=2 ** 20, k_ld=2 ** 20, v_ld=2 ** 20), 1),
    (dict(B=0, q=None, cu_seqlens=None), 0), (dict(T=0, q=None, k=None, v=None, out=None), 0)])
def test_prompt_arguments(kw, rc):
    assert prompt(**kw) == rc
    assert tps.load().tps_prompt_attention(None, None) == 1


def test_prompt_stall_test_hook_checks_its_wait_limit():
    a = decode._Prompt(B=0, n_q_heads=4, n_k_heads=4, head_dim=64, scale=1.0)
    for wait, rc in ((0, 1), (10 ** 9 + 1, 1), (1, 0), (10 ** 9, 0)):
        assert tps.load().tps_prompt_attention_stall_test(ctypes.byref(a), 0, wait, None) == rc


def test_binding_refuses_tensors_that_are_not_on_a_gpu():
    x = torch.zeros(2, 4, 64).bfloat16()
    with pytest.raises(ValueError):
        tps.prompt_attention(x, x, x, torch.zeros(2, dtype=torch.int32))


def pages(**kw):
    a = dict(page_table=FAKE, seq_len=FAKE, change=FAKE, free_pages=FAKE, free_count=FAKE, B=3, table_width=4, table_ld=4, n_free=9, page_size=16)
    a.update(kw)
    return decode._Pages(**a)


def extend(tokens=5, slots=FAKE, positions=FAKE, cu=FAKE, **kw):
    v = ctypes.c_void_p
    return tps.load().tps_kv_extend(ctypes.byref(pages(**kw)), tokens, v(slots), v(positions), v(cu), None)


@pytest.mark.parametrize("kw,rc", [
    (dict(page_table=None), 1), (dict(seq_len=None), 1), (dict(change=None), 1), (dict(free_pages=None), 1), (dict(free_count=None), 1), (dict(B=-1), 1),
    (dict(B=2 ** 31), 1), (dict(table_width=-1), 1), (dict(table_ld=3), 1), (dict(table_width=2 ** 27, table_ld=2 ** 27), 1), (dict(n_free=-1), 1),
    (dict(n_free=2 ** 31), 1), (dict(page_size=8), 1), (dict(page_size=48), 1), (dict(page_size=512), 1), (dict(page_table=FAKE + 2), 4),
    (dict(seq_len=FAKE + 1), 4), (dict(change=FAKE + 2), 4), (dict(free_pages=FAKE + 2), 4), (dict(free_count=FAKE + 2), 4), (dict(out_status=FAKE + 1), 4)])
def test_pages_arguments(kw, rc):
    assert extend(**kw) == rc
    assert tps.load().tps_kv_trim(ctypes.byref(pages(**kw)), None) == rc


def test_extend_and_trim_arguments():
    for kw, rc in ((dict(tokens=-1), 1), (dict(tokens=2 ** 31), 1), (dict(slots=None), 1), (dict(positions=None), 1), (dict(cu=None), 1),
                   (dict(slots=FAKE + 4), 4), (dict(positions=FAKE + 2), 4), (dict(cu=FAKE + 2), 4)):
        assert extend(**kw) == rc
    assert tps.load().tps_kv_extend(None, 0, None, None, ctypes.c_void_p(FAKE), None) == 1
    assert tps.load().tps_kv_trim(None, None) == 1
    assert tps.load().tps_kv_trim(ctypes.byref(pages(B=0, page_table=None, seq_len=None, change=None)), None) == 0


def cache(**kw):
    a = dict(k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, n_pages=4, n_heads=2, page_size=16, head_dim=64, format=1)
    a.update(kw)
    return decode._Cache(**a)


def tree(c=None, **kw):
    a = dict(q=FAKE, out=FAKE, page_table=FAKE, seq_len=FAKE, tree=FAKE, B=3, table_width=2, table_ld=2, tree_ld=5, n_nodes=5, n_q_heads=4, scale=1.0)
    a.update(kw)
    return tps.load().tps_tree_attention(ctypes.byref(c or cache()), ctypes.byref(decode._Tree(**a)), None)


@pytest.mark.parametrize("kw,rc", [
    (dict(B=-1), 1), (dict(table_width=-1, table_ld=0), 1), (dict(table_ld=1), 1), (dict(table_width=2 ** 27, table_ld=2 ** 27), 1), (dict(n_nodes=0), 1),
    (dict(n_nodes=65, tree_ld=65), 1), (dict(tree_ld=4), 1), (dict(n_q_heads=0), 1), (dict(n_q_heads=3), 1), (dict(n_q_heads=2 ** 16), 1),
    (dict(scale=float("nan")), 1), (dict(scale=-3e38), 1), (dict(q=None), 1), (dict(out=None), 1), (dict(page_table=None), 1), (dict(seq_len=None), 1), (dict(tree=None), 1),
    (dict(q=FAKE + 8), 4), (dict(out=FAKE + 8), 4), (dict(out_lse=FAKE + 2), 4), (dict(page_table=FAKE + 2), 4), (dict(seq_len=FAKE + 2), 4),
    (dict(tree_len=FAKE + 2), 4), (dict(tree=FAKE + 4), 4), (dict(out_status=FAKE + 2), 4), (dict(workspace=FAKE + 128), 4),
    (dict(B=0, q=None, tree=None), 0)])
def test_tree_arguments(kw, rc):
    assert tree(**kw) == rc


@pytest.mark.parametrize("kw,rc", [(dict(k=None), 1), (dict(v_scale=None), 1), (dict(format=3), 1), (dict(page_size=8), 1), (dict(head_dim=96), 1),
                                   (dict(n_heads=0), 1), (dict(v=FAKE + 8), 4)])
def test_tree_caches(kw, rc):
    assert tree(c=cache(**kw)) == rc


def test_tree_workspace_and_stall_test_hook():
    lib, c = tps.load(), cache()
    assert lib.tps_tree_attention_workspace(ctypes.byref(c), ctypes.byref(decode._Tree(n_nodes=0))) == -1
    assert lib.tps_tree_attention_workspace(ctypes.byref(c), None) == -1
    a = decode._Tree(B=0, n_nodes=4, n_q_heads=4, scale=1.0)
    assert lib.tps_tree_attention_workspace(ctypes.byref(c), ctypes.byref(a)) == 0
    assert lib.tps_tree_attention(None, ctypes.byref(a), None) == 1 and lib.tps_tree_attention(ctypes.byref(c), None, None) == 1
    for wait, rc in ((0, 1), (10 ** 9 + 1, 1), (1, 0), (10 ** 9, 0)):
        assert lib.tps_tree_attention_stall_test(ctypes.byref(c), ctypes.byref(a), 0, wait, None) == rc


def test_row_status_text():
    assert b"pages" in tps.load().tps_status_string(105)
