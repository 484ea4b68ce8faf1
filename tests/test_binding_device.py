"""Every call of the binding launches on its tensors' device, whichever is current
(the library launches on the current device): on the CPU, with the library and the
device switch replaced by ones that record.
"""
import contextlib

import pytest
import torch

import mla_latent_decode_gb300 as mla

bf, i32, u8 = torch.bfloat16, torch.int32, torch.uint8


def z(*shape, dtype=bf):
    return torch.zeros(shape, dtype=dtype)


CALLS = {
    "lse_combine": lambda: mla.lse_combine(z(2, 3, 512, dtype=torch.float32), z(2, 3, dtype=torch.float32)),
    "lse_combine_bf16": lambda: mla.lse_combine(z(2, 3, 512), z(2, 3, dtype=torch.float32)),
    "kv_write": lambda: mla.kv_write(z(4, 576), z(4, dtype=i32), z(64, 576)),
    "absorb_q": lambda: mla.absorb_q(z(1, 1, 2, 128), z(2, 128, 512)),
    "project_out": lambda: mla.project_out(z(1, 1, 2, 512), z(2, 512, 128)),
    "kv_append": lambda: mla.kv_append(z(4, 576), z(4, dtype=i32), z(4, dtype=i32), z(8, 64, dtype=torch.float32), z(64, 576)),
    "kv_read": lambda: mla.kv_read(z(64, 576), z(4, dtype=i32)),
    "add_rms_norm": lambda: mla.add_rms_norm(z(2, 64), z(64)),
    "decode_partial": lambda: mla.decode_partial(z(1, 1, 2, 512), z(1, 1, 2, 64), z(64, 576), None, z(1, 64, dtype=i32),
                                                 z(1, dtype=i32), None, 1, 0.07),
    "debug_gather": lambda: mla.debug_gather(z(64, 576), z(1, 64, dtype=i32), z(1, dtype=i32), z(2, dtype=i32), 1),
}


@pytest.mark.parametrize("name", CALLS)
def test_launches_on_the_tensors_device(name, monkeypatch):
    inside, seen = [], []

    @contextlib.contextmanager
    def on(t):
        inside.append(t.device)
        yield
        inside.pop()

    class Library:
        def __getattr__(self, fn):
            return lambda *args: seen.append(list(inside)) or 0

    monkeypatch.setattr(mla, "_on", on)
    monkeypatch.setattr(mla, "_stream", lambda stream: seen.append(list(inside)))
    monkeypatch.setattr(mla, "library", lambda: Library())
    CALLS[name]()
    assert len(seen) == 2  # the stream is looked up and the kernel launched, both there
    assert all(where == [torch.device("cpu")] for where in seen)
