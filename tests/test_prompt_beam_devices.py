"""The prompts', beams' and pages' entry points refuse an array that is on another device
than the first one (a length or a score left on the host): the kernels read them by
address.  On the CPU the other device is an array that says so."""
import pytest
import torch

import mla_latent_decode_gb300 as mla

bf, f32, i32, u8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


class Elsewhere(torch.Tensor):
    def get_device(self):
        return 3

    @property
    def device(self):
        return torch.device("cuda", 3)


class Library:
    def __getattr__(self, fn):
        return lambda *args: 0


def _calls(dev):
    def z(*shape, dtype=i32):
        return torch.zeros(shape, dtype=dtype, device=dev)

    return {
        "prefill": (mla.prefill, "q_nope", dict(
            q_nope=z(5, 2, 128, dtype=bf), q_rope=z(5, 2, 64, dtype=bf), k_nope=z(7, 2, 128, dtype=bf), k_rope=z(7, 64, dtype=bf),
            v=z(7, 2, 128, dtype=bf), cu_q=z(2), cu_kv=z(2), work=z(1, 8), sm_scale=0.07, prefix=z(1), num_parts=1,
            O_part=z(1, 2, 256, 128, dtype=f32), LSE_part=z(1, 2, 256, dtype=f32), out=z(5, 2, 128, dtype=bf),
            lse_out=z(5, 2, dtype=f32), status=z(1))),
        "beam_select": (mla.beam_select, "logits", dict(
            logits=z(2, 3, 50, dtype=bf), scores=z(2, 3, dtype=f32), k=4, finished=z(2, 3, dtype=u8), out_scores=z(2, 4, dtype=f32),
            parents=z(2, 4), tokens=z(2, 4), status=z(1))),
        "pages_fork": (mla.pages_fork, "table", dict(
            table=z(2, 128), lens=z(2), refs=z(9), free_count=z(1), parents=z(2), keep=z(2), grow=z(2), table_out=z(2, 128),
            lens_out=z(2), copies=z(3, 2), status=z(1))),
        "pages_compact": (mla.pages_compact, "table", dict(
            table=z(2, 128), lens=z(2), refs=z(9), max_moves=3, table_out=z(2, 128), src=z(3), dst=z(3), count=z(1), status=z(1))),
        "kv_copy": (mla.kv_copy, "kv", dict(
            kv=z(128, 576, dtype=u8), src=z(2), dst=z(2), kv_scale=z(128, dtype=f32), tokens=z(2), count=z(1), status=z(1))),
    }


CASES = [(name, arg) for name, (_, first, args) in _calls("cpu").items()
         for arg, x in args.items() if torch.is_tensor(x) and arg != first]


@pytest.fixture
def no_launch(monkeypatch):
    monkeypatch.setattr(mla, "_launch", lambda *args: None)
    monkeypatch.setattr(mla, "library", lambda: Library())


@pytest.mark.parametrize("name,arg", CASES)
def test_an_array_elsewhere_is_refused(name, arg, no_launch):
    fn, _, args = _calls("cpu")[name]
    fn(**args)
    with pytest.raises(ValueError, match=f"^{arg}: "):
        fn(**{**args, arg: args[arg].as_subclass(Elsewhere)})


@pytest.mark.gpu
@pytest.mark.parametrize("name,arg", CASES)
def test_an_array_on_the_host_is_refused(name, arg, no_launch):
    fn, _, args = _calls("cuda")[name]
    fn(**args)
    with pytest.raises(ValueError, match=f"^{arg}: "):
        fn(**{**args, arg: args[arg].cpu()})
