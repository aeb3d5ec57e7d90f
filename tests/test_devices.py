"""Every call looks where all its tensors are, those that a kernel writes among
them, and at the stream, before it takes a pointer.  CPU only."""
import pytest

import paged_kv_cache_num_gb300 as pkv


class On:
    """What says where it is, and nothing else."""

    def __init__(self, dev):
        self.dev = dev

    def get_device(self):
        return self.dev


class Stream:
    device_index = 1


def cache(dev=0):
    return pkv.KVCache("f16", On(dev), On(dev))


A = lambda: On(0)  # noqa: E731
CALLS = {
    "slot_mapping": (lambda **k: pkv.slot_mapping(A(), A(), A(), 16, **k), ("out", "err_flag")),
    "kv_append": (lambda cache=None, **k: pkv.kv_append(A(), A(), A(), cache or globals()["cache"](), **k), ("err_flag",)),
    "kv_append_scaled": (lambda cache=None, **k: pkv.kv_append_scaled(A(), A(), A(), A(), A(), cache or globals()["cache"](), **k), ("err_flag",)),
    "kv_append_dynamic": (lambda cache=None, **k: pkv.kv_append_dynamic(A(), A(), A(), cache or globals()["cache"](), **k), ("err_flag",)),
    "kv_gather": (lambda cache=None, **k: pkv.kv_gather(cache or globals()["cache"](), A(), **k), ("k_out", "v_out", "err_flag")),
    "paged_decode": (lambda cache=None, **k: pkv.paged_decode(A(), cache or globals()["cache"](), A(), A(), **k), ("out", "workspace", "err_flag")),
    "decode_step": (lambda cache=None, **k: pkv.decode_step(A(), A(), A(), A(), A(), cache or globals()["cache"](), A(), A(), **k),
                    ("out", "slots", "workspace", "err_flag")),
    "paged_decode_noalloc": (lambda cache=None, **k: pkv.paged_decode_noalloc(A(), cache or globals()["cache"](), A(), A(), **k), ("out", "err_flag")),
    "paged_prefill": (lambda cache=None, **k: pkv.paged_prefill(A(), cache or globals()["cache"](), A(), A(), A(), **k), ("out", "workspace", "err_flag")),
    "norm_rope": (lambda **k: pkv.norm_rope(A(), A(), A(), A(), **k), ("q_weight", "k_weight", "q_out", "k_out", "err_flag")),
    "norm_rope_append": (lambda cache=None, **k: pkv.norm_rope_append(A(), A(), A(), A(), A(), A(), cache or globals()["cache"](), **k),
                         ("q_weight", "k_weight", "q_out", "err_flag")),
    "extend_tables": (lambda **k: pkv.extend_tables(A(), A(), A(), A(), A(), 16, **k),
                      ("context_lens", "q_starts", "req", "pos", "slot_mapping", "free_left", "err_flag")),
    "trim_tables": (lambda **k: pkv.trim_tables(A(), A(), A(), A(), A(), 16, **k), ("kept_lens", "free_left", "err_flag")),
    "pack3": (lambda **k: pkv.pack3(A(), **k), ("packed",)),
    "unpack3": (lambda **k: pkv.unpack3(A(), **k), ("values",)),
    "unpack3_words": (lambda **k: pkv.unpack3_words(A(), **k), ("values",)),
    "copy_peak": (lambda dst=None, **k: pkv.copy_peak(A(), dst or A(), **k), ("dst",)),
}
EACH = [(n, a) for n, (_, args) in CALLS.items() for a in args]


@pytest.mark.parametrize("name,arg", EACH)
def test_tensors_elsewhere(name, arg):
    call = CALLS[name][0]
    with pytest.raises(ValueError, match="CUDA tensors"):
        call(**{arg: On(-1)})                     # on the CPU
    with pytest.raises(ValueError, match="one device"):
        call(**{arg: On(1)})


@pytest.mark.parametrize("name", [n for n, c in CALLS.items() if "cache" in c[0].__code__.co_varnames])
def test_caches_elsewhere(name):
    with pytest.raises(ValueError, match="one device"):
        CALLS[name][0](cache=cache(1))


@pytest.mark.parametrize("name", list(CALLS))
def test_streams_elsewhere(name):
    with pytest.raises(ValueError, match="the stream is on cuda:1"):
        CALLS[name][0](stream=Stream())
