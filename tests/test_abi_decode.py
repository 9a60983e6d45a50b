"""The decode-step entry points reject bad arguments before anything reaches the GPU, in the C ABI and
in the binding."""
import ctypes
import os
import subprocess
import sys
import threading
import time

import pytest
import torch

import nucleus_token_sampler_gb300 as tps
from nucleus_token_sampler_gb300 import decode

FAKE = 0x10000  # never dereferenced: every call below fails validation first, or has nothing to do


def norm(**kw):
    a = dict(q=FAKE, k=FAKE, out_q=FAKE, out_k=FAKE, q_ld=512, q_hd=128, k_ld=512, k_hd=128, oq_ld=512, oq_hd=128, ok_ld=512,
             ok_hd=128, positions=FAKE, cos_sin=FAKE, T=2, n_positions=10, n_q_heads=4, n_k_heads=4, head_dim=128,
             rot_dim=128, interleaved=0, dtype=0, eps=1e-6)
    a.update(kw)
    return tps.load().tps_qk_norm_rope(ctypes.byref(decode._NormRope(**a)), None)


@pytest.mark.parametrize("kw,rc", [
    (dict(T=-1), 1), (dict(n_q_heads=-1), 1), (dict(n_k_heads=65536), 1), (dict(head_dim=0), 1), (dict(head_dim=8193), 1),
    (dict(rot_dim=129), 1), (dict(rot_dim=3), 1), (dict(rot_dim=-2), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
    (dict(eps=float("inf")), 1), (dict(q=None), 1), (dict(out_k=None), 1), (dict(positions=None), 1), (dict(cos_sin=None), 1),
    (dict(n_positions=-1), 1), (dict(dtype=5), 2), (dict(q=FAKE + 2), 4), (dict(k=FAKE + 1, dtype=1), 4),
    (dict(positions=FAKE + 2), 4), (dict(q_weight=FAKE + 1), 4), (dict(out_status=FAKE + 3), 4),
    (dict(T=0), 0), (dict(n_q_heads=0, n_k_heads=0), 0)])
def test_norm_rope_arguments(kw, rc):
    assert norm(**kw) == rc
    assert tps.load().tps_qk_norm_rope(None, None) == 1


def cache(**kw):
    a = dict(k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, n_pages=4, n_heads=2, page_size=16, head_dim=64, format=1)
    a.update(kw)
    return decode._Cache(**a)


BAD_CACHES = [(dict(k=None), 1), (dict(v=None), 1), (dict(k_scale=None), 1), (dict(format=3), 1), (dict(format=-1), 1),
              (dict(page_size=8), 1), (dict(page_size=24), 1), (dict(page_size=512), 1), (dict(head_dim=24), 1), (dict(head_dim=528), 1),
              (dict(head_dim=0), 1), (dict(n_heads=0), 1), (dict(n_pages=0), 1), (dict(n_pages=1 << 31), 1), (dict(k=FAKE + 8), 4),
              (dict(v_scale=FAKE + 2), 4)]


@pytest.mark.parametrize("kw,rc", BAD_CACHES)
def test_cache_arguments(kw, rc):
    lib, v = tps.load(), ctypes.c_void_p(FAKE)
    c = cache(**kw)
    assert lib.tps_kv_write(ctypes.byref(c), v, v, 0, 4, 128, 64, 128, 64, v, None) == rc
    assert lib.tps_kv_read(ctypes.byref(c), v, 4, v, v, 0, None) == rc
    assert attention(c=c) == rc


def test_write_and_read_arguments():
    lib, v, c = tps.load(), ctypes.c_void_p, cache()

    def write(k=FAKE, x=FAKE, dtype=0, T=4, slots=FAKE, c=c):
        return lib.tps_kv_write(ctypes.byref(c), v(k), v(x), dtype, T, 128, 64, 128, 64, v(slots), None)

    def read(k=FAKE, x=FAKE, dtype=0, T=4, slots=FAKE):
        return lib.tps_kv_read(ctypes.byref(c), v(slots), T, v(k), v(x), dtype, None)
    for f in (write, read):
        assert f(T=-1) == 1 and f(k=None) == 1 and f(x=None) == 1 and f(slots=None) == 1
        assert f(dtype=2) == 2
        assert f(k=FAKE + 2) == 4 and f(slots=FAKE + 4) == 4
        assert f(T=0, k=None, x=None, slots=None) == 0
    assert write(c=cache(format=0, k_scale=None, v_scale=None), T=0) == 0
    assert lib.tps_kv_write(None, v(FAKE), v(FAKE), 0, 4, 128, 64, 128, 64, v(FAKE), None) == 1
    assert lib.tps_kv_read(None, v(FAKE), 4, v(FAKE), v(FAKE), 0, None) == 1


def attention(c=None, **kw):
    a = dict(q=FAKE, out=FAKE, prefix_pages=FAKE, page_table=FAKE, suffix_len=FAKE, B=3, prefix_len=40, table_width=2,
             table_ld=2, q_len=1, n_q_heads=4, scale=1.0)
    a.update(kw)
    return tps.load().tps_prefix_attention(ctypes.byref(c or cache()), ctypes.byref(decode._Attention(**a)), None)


@pytest.mark.parametrize("kw,rc", [
    (dict(B=-1), 1), (dict(prefix_len=-1), 1), (dict(prefix_len=1 << 31), 1), (dict(table_width=-1, table_ld=0), 1),
    (dict(table_ld=1), 1), (dict(q_len=0), 1), (dict(n_q_heads=0), 1), (dict(n_q_heads=3), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(q=None), 1), (dict(out=None), 1), (dict(suffix_len=None), 1),
    (dict(prefix_pages=None), 1), (dict(page_table=None), 1), (dict(q=FAKE + 8), 4), (dict(out=FAKE + 2), 4),
    (dict(out_lse=FAKE + 2), 4), (dict(suffix_len=FAKE + 2), 4), (dict(workspace=FAKE + 16), 4), (dict(B=0, q=None), 0)])
def test_attention_arguments(kw, rc):
    assert attention(**kw) == rc


def test_attention_head_sizes_and_null_structs():
    lib = tps.load()
    assert attention(c=cache(head_dim=96)) == 1 and attention(c=cache(head_dim=256)) == 1
    assert lib.tps_prefix_attention(None, ctypes.byref(decode._Attention()), None) == 1
    assert lib.tps_prefix_attention(ctypes.byref(cache()), None, None) == 1
    assert lib.tps_prefix_attention_workspace(ctypes.byref(cache()), ctypes.byref(decode._Attention(q_len=0))) == -1
    none = decode._Attention(B=0, q_len=1, n_q_heads=4, scale=1.0)
    assert lib.tps_prefix_attention_workspace(ctypes.byref(cache()), ctypes.byref(none)) == 0


def test_binding_refuses_tensors_that_are_not_on_a_gpu():
    x = torch.zeros(2, 4, 64)
    with pytest.raises(ValueError):
        tps.qk_norm_rope(x, x, None, None, torch.zeros(2, dtype=torch.int32), torch.zeros(4, 64))
    with pytest.raises(ValueError):
        tps.KVCache(torch.zeros(2, 2, 16, 64, dtype=torch.int8), torch.zeros(2, 2, 16, 64, dtype=torch.int8))
    with pytest.raises(ValueError):
        tps.KVCache.empty(2, 2, 16, 64, "int4")
    with pytest.raises(ValueError):
        tps.prefix_attention(x.bfloat16(), None, None, 0, None, None)


def test_first_use_from_two_threads_finds_the_module_bound(monkeypatch):
    """The native module's entry points are null until `bind` has run: no thread may get hold of it before."""
    class Slow:
        def __init__(self):
            self.bound = False

        def bind(self, *args):
            time.sleep(0.05)
            self.bound = True
    made = []

    def load_binding():
        made.append(Slow())
        return made[-1]
    monkeypatch.setattr(tps, "load_binding", load_binding)
    monkeypatch.setattr(decode, "_ops", None)
    seen = []

    def use():
        ops = decode._ops or decode._torch_ops()  # as every call begins
        seen.append(ops.bound)
    threads = [threading.Thread(target=use) for _ in range(8)]
    for t in threads:
        t.start()
        time.sleep(0.01)
    for t in threads:
        t.join()
    assert seen == [True] * 8 and len(made) == 1


def test_the_native_module_refuses_calls_before_it_is_bound():
    code = ("import nucleus_token_sampler_gb300 as tps\n"
            "ops = tps.load_binding()\n"
            "for f in (ops.norm, ops.write, ops.read, ops.attention):\n"
            "    try:\n"
            "        f()\n"
            "    except RuntimeError as e:\n"
            "        assert 'bound' in str(e), e\n"
            "    else:\n"
            "        raise AssertionError('not refused')\n")
    subprocess.run([sys.executable, "-c", code], check=True, cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


def test_stall_test_hook_of_the_attention_checks_its_wait_limit():
    lib = tps.load()
    a = decode._Attention(B=0, q_len=1, n_q_heads=4, scale=1.0)
    for wait, rc in ((0, 1), (10 ** 9 + 1, 1), (1, 0), (10 ** 9, 0)):
        assert lib.tps_prefix_attention_stall_test(ctypes.byref(cache()), ctypes.byref(a), 0, wait, None) == rc


@pytest.mark.parametrize("page", [16, 256])
def test_attention_refuses_lengths_whose_token_numbers_would_pass_32_bits(page):
    """A walk counts tokens in 32 bits and goes on by up to 512 past the last one."""
    most, c = 2 ** 31 - 2 ** 16, cache(page_size=page)
    lib, wide = tps.load(), most // page

    def size(**kw):
        a = dict(B=1, prefix_len=40, table_width=2, table_ld=2, q_len=1, n_q_heads=2, scale=1.0)
        a.update(kw)
        return lib.tps_prefix_attention_workspace(ctypes.byref(c), ctypes.byref(decode._Attention(**a)))
    for kw in (dict(prefix_len=most + 1), dict(prefix_len=2 ** 31 - 1), dict(table_width=wide + 1, table_ld=wide + 1),
               dict(table_width=2 ** 31 - 1, table_ld=2 ** 31 - 1)):
        assert attention(c=c, **kw) == 1 and size(**kw) == -1
    assert attention(c=c, B=0, prefix_len=most, table_width=wide, table_ld=wide) == 0


@pytest.mark.parametrize("name", ["k", "v", "k_scale", "v_scale"])
def test_a_cache_keeps_the_tensors_it_was_made_with(name):
    """The calls go to the addresses these tensors had: another tensor in their place would leave freed memory written to."""
    c = tps.KVCache.__new__(tps.KVCache)
    with pytest.raises(AttributeError):
        setattr(c, name, torch.zeros(1))
