"""Flags, workspaces and byte buffers that a kernel would write beyond are refused
before any launch.  CPU only: the device checks are taken out and the library is
replaced by one that must not be called."""
import pytest
import torch

from paged_kv_cache_num_gb300 import pkv

KV = torch.zeros((4, 16, 2, 64), dtype=torch.float16)
X = torch.zeros((3, 2, 64), dtype=torch.float16)
I = torch.zeros(3, dtype=torch.int32)      # noqa: E741
BT = torch.zeros((3, 2), dtype=torch.int32)
U8 = torch.zeros(64, dtype=torch.uint8)


class Lib:
    def __getattr__(self, name):
        def call(*args):
            raise AssertionError("%s was called" % name)
        return call


@pytest.fixture(autouse=True)
def no_device(monkeypatch):
    monkeypatch.setattr(pkv, "_one_device", lambda *ts: 0)
    monkeypatch.setattr(pkv, "_elsewhere", lambda dev, stream: None)
    monkeypatch.setattr(pkv, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(pkv, "lib", Lib)


def cache():
    return pkv.KVCache("f16", KV, KV.clone())


CALLS = {
    "slot_mapping": lambda **k: pkv.slot_mapping(BT, I, I, 16, **k),
    "kv_append": lambda **k: pkv.kv_append(X, X, I.long(), cache(), **k),
    "kv_append_scaled": lambda **k: pkv.kv_append_scaled(X, X, X.float()[..., 0], X.float()[..., 0], I.long(), cache(), **k),
    "kv_append_dynamic": lambda **k: pkv.kv_append_dynamic(X, X, I.long(), cache(), **k),
    "kv_gather": lambda **k: pkv.kv_gather(cache(), I.long(), **k),
    "paged_decode": lambda workspace=U8, **k: pkv.paged_decode(X, cache(), BT, I, workspace=workspace, **k),
    "decode_step": lambda workspace=U8, **k: pkv.decode_step(X, X, I, I, X, cache(), BT, I, workspace=workspace, **k),
    "paged_decode_noalloc": lambda **k: pkv.paged_decode_noalloc(X, cache(), BT, I, **k),
    "paged_prefill": lambda workspace=U8, **k: pkv.paged_prefill(X, cache(), BT, torch.zeros(4, dtype=torch.int32), I, workspace=workspace, **k),
    "norm_rope": lambda **k: pkv.norm_rope(X, X, torch.zeros((4, 32)), I, **k),
    "norm_rope_append": lambda **k: pkv.norm_rope_append(X, X, X, torch.zeros((4, 32)), I, I.long(), cache(), **k),
    "extend_tables": lambda **k: pkv.extend_tables(BT, I, I, I, I[:1], 16, 4, **k),
    "trim_tables": lambda **k: pkv.trim_tables(BT, I, I, I, I[:1], 16, **k),
}


@pytest.mark.parametrize("name", list(CALLS))
@pytest.mark.parametrize("flag", [torch.zeros(1, dtype=torch.uint8), torch.zeros(1, dtype=torch.int64), torch.zeros(1), torch.zeros(0, dtype=torch.int32)])
def test_flags(name, flag):
    with pytest.raises(ValueError, match="err_flag"):
        CALLS[name](err_flag=flag)


@pytest.mark.parametrize("name", ["paged_decode", "decode_step", "paged_prefill"])
@pytest.mark.parametrize("space", [torch.zeros(1, dtype=torch.uint8).expand(1 << 20), torch.zeros((8, 64), dtype=torch.uint8)[:, :16]])
def test_workspaces(name, space):
    with pytest.raises(ValueError, match="workspace"):
        CALLS[name](workspace=space)


def test_bytes():
    u8 = lambda n: torch.zeros(n, dtype=torch.uint8)  # noqa: E731
    for call in (lambda: pkv.pack3(u8(32), u8(11)), lambda: pkv.pack3(u8(64)[::2], u8(12)), lambda: pkv.unpack3(u8(12), u8(31)),
                 lambda: pkv.unpack3(u8(12), u8(64)[::2]), lambda: pkv.unpack3_words(torch.zeros(6, dtype=torch.int32), u8(63)),
                 lambda: pkv.unpack3_words(torch.zeros(6, dtype=torch.int16), u8(64)), lambda: pkv.copy_peak(u8(64), u8(48))):
        with pytest.raises(ValueError, match="bytes or more"):
            call()
