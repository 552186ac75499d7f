"""The row calls and calls over int8 pools without a GPU: sizes whose products leave their integers, tensors of another device,
empty batches, and a step that checked mode refuses."""
import pytest
import torch

import paged_kv_cache_409_b200 as pkv
from paged_kv_cache_409_b200 import _binding
from test_binding_marshalling import mock  # noqa: F401

EINVAL, EUNSUPPORTED = -1, -2
P = 1 << 20


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_409_b200 import build
    build.build()
    return pkv.load_library()


def test_block_bytes_beyond_64_bits_are_refused(lib):
    big = 2**31 - 1
    for sizes in ((2**30, 2**30, 2**30), (big, big, big), (big, big, 1), (2**30, 2**30, 4)):
        b, h, d = sizes
        assert lib.pkv_int8_block_bytes(b, h, d) == (b * h * (d + 4) if b * h * (d + 4) < 2**63 else EINVAL), sizes
    assert lib.pkv_int8_block_bytes(2**30, 2, 2**30) == 2**31 * (2**30 + 4)


def test_pools_of_uncountable_slots_are_refused(lib):
    for fn in (lib.pkv_reshape_and_cache_int8, lib.pkv_read_cache_int8):
        assert fn(P, P, P, P, P, 0, 2, 64, 16, 2**63 // 16 - 1, 1, None) == 0
        assert fn(P, P, P, P, P, 0, 2, 64, 16, 2**63 // 16, 1, None) == EINVAL
        assert fn(P, P, P, P, P, 0, 2**31 - 4, 64, 2**31 - 4, 4, 1, None) == EUNSUPPORTED

    def rope(fn, blocks):
        return fn(P, P, P, P, 512, 128, 128, 0, 0, 1e-6, P, 9, 64, 0, P, P, P, P, 0, 8, 2, 64, 16, blocks, 1, *tail, None)

    for fn, tail in ((lib.pkv_rope_and_cache, ()), (lib.pkv_rope_and_cache_fp8, (1.0, 1.0)), (lib.pkv_rope_and_cache_int8, ())):
        assert rope(fn, 2**63 // 16 - 1) == 0 and rope(fn, 2**63 // 16) == EINVAL


def test_checked_mode_without_host_memory_is_an_error():
    """PKV_CHECK=1 copies the tables to the host: when there is no memory for that, the call fails, and the process goes on."""
    import subprocess
    import sys

    from paged_kv_cache_409_b200 import build
    code = f"""
import ctypes, os, resource
os.environ['PKV_CHECK'] = '1'
lib = ctypes.CDLL({build.build()!r})
resource.setrlimit(resource.RLIMIT_AS, (4 << 30, 4 << 30))
I, L, V = ctypes.c_int, ctypes.c_int64, ctypes.c_void_p
P = V({P})
n = L(2**31 - 1)  # 16 GiB of slots
args = [P, P, P, P, P, n, I(2), I(64), I(16), L(4), I(1)]
for name in ('pkv_reshape_and_cache_int8', 'pkv_read_cache_int8', 'pkv_reshape_and_cache'):
    assert getattr(lib, name)(*args, V()) == -4, name
lib.pkv_last_cuda_error.restype = ctypes.c_char_p
assert b'memory' in lib.pkv_last_cuda_error()
print('refused')
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=200)
    assert r.returncode == 0 and "refused" in r.stdout, (r.returncode, r.stdout + r.stderr)


class Elsewhere(torch.Tensor):
    """A tensor that says it lies on another device than the call's other ones."""

    def get_device(self):
        return 5


def test_pools_of_another_device_are_refused(mock, monkeypatch):  # noqa: F811
    monkeypatch.setattr(_binding, "_current_device", lambda: 0)
    T, Hq, H, D = 2, 4, 2, 64
    q, k, i = torch.zeros(T, Hq, D).half(), torch.zeros(T, H, D).half(), torch.zeros(T, dtype=torch.int64)
    for call, pool, tail in ((pkv.rope_and_cache, torch.zeros(4, 16, H, D).half(), ()),
                             (pkv.rope_and_cache_fp8, torch.zeros(4, 16, H, D, dtype=torch.uint8), (1.0, 1.0)),
                             (pkv.rope_and_cache_int8, torch.zeros(4, 16, H, D + 4, dtype=torch.uint8), ())):
        call(q, q, k, k, None, None, pool, pool, i, *tail)
        for pools in ((pool.as_subclass(Elsewhere), pool), (pool, pool.as_subclass(Elsewhere))):
            with pytest.raises(ValueError):
                call(q, q, k, k, None, None, *pools, i, *tail)
        for bad in (dict(cos_sin=torch.zeros(9, 32).as_subclass(Elsewhere), positions=i),
                    dict(cos_sin=torch.zeros(9, 32), positions=i.as_subclass(Elsewhere)),
                    dict(cos_sin=None, positions=None, q_norm_weight=torch.zeros(D).half().as_subclass(Elsewhere))):
            with pytest.raises(ValueError):
                call(q, q, k, k, key_cache=pool, value_cache=pool, slot_mapping=i, **bad,
                     **dict(zip(("k_scale", "v_scale"), tail)))


def test_an_empty_batch_of_any_layout_passes(mock):  # noqa: F811
    """No token: whatever the strides of the empty rows are, with tables and weights given."""
    Hq, H, D = 4, 2, 64
    q, k, i = torch.zeros(0, D, Hq).half().transpose(1, 2), torch.zeros(0, D, H).half().transpose(1, 2), torch.zeros(0, dtype=torch.int64)
    pool, w, table = torch.zeros(4, 16, H, D).half(), torch.zeros(D).half(), torch.zeros(9, 32)
    pkv.rope_and_cache(torch.zeros(0, Hq, D).half(), q, k, k, table, i, pool, pool, i, q_norm_weight=w, k_norm_weight=w)
    name, a = mock.last()
    assert name == "pkv_rope_and_cache"
    assert (a["num_tokens"], a["q_norm_weight"], a["k_norm_weight"], a["cos_sin"], a["rotary_dim"], a["max_position"]) == (
        0, w.data_ptr(), w.data_ptr(), table.data_ptr(), 32, 9)
