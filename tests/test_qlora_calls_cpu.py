"""What the adapter layer does on the host before and around its launches, with
the library's calls and the device replaced by stand-ins."""

import contextlib

import pytest
import torch

from bit_grouped_moe_e4b_b200 import e4b, qlora

E, H, I, R1, R2, T, K = 2, 64, 128, 8, 16, 3, 2


@pytest.fixture
def calls(monkeypatch):
    """Names of the library's calls, each with the device that was current."""
    seen, current = [], [None]

    @contextlib.contextmanager
    def device(d):
        before, current[0] = current[0], torch.device(d)
        yield
        current[0] = before

    monkeypatch.setattr(qlora.torch.cuda, "device", device)
    for name in ("e4b_route", "e4b_permute", "e4b_permute_backward", "e4b_unpermute", "e4b_unpermute_backward",
                 "e4b_glu_backward", "e4b_lora", "e4b_lora_backward", "e4b_grouped_gemm", "e4b_grouped_dgrad"):
        monkeypatch.setattr(e4b, name, lambda *a, _n=name, **kw: seen.append((_n, current[0])))
    return seen


def inputs(dtype=torch.int32, T=T):
    layer = e4b.PackedLayer("nf4", E, H, I, *[torch.zeros(1)] * 4)
    ads = [qlora.Adapter(torch.zeros(E, R1, H), torch.zeros(E, 2 * I, R1)),
           qlora.Adapter(torch.zeros(E, R2, I), torch.zeros(E, H, R2))]
    return layer, ads, torch.zeros(T, H, dtype=torch.bfloat16), torch.zeros(T, K, dtype=dtype), torch.zeros(T, K)


def test_every_call_runs_on_the_tensors_device(calls):
    layer, ads, x, ids, gates = inputs()
    y, kept = qlora.forward(layer, *ads, x, ids, gates)
    assert [n for n, _ in calls] == ["e4b_route", "e4b_permute", "e4b_grouped_gemm", "e4b_lora", "e4b_grouped_gemm",
                                     "e4b_lora", "e4b_unpermute"]
    qlora.backward(layer, *ads, kept, torch.zeros_like(x))
    assert len(calls) == 14 and all(d == x.device for _, d in calls)


def test_ids_of_another_type_or_batch_are_refused(calls):
    layer, ads, x, _, gates = inputs()
    for bad in (torch.zeros(T, K, dtype=torch.int64), torch.zeros(T, K), torch.zeros(T + 1, K, dtype=torch.int32),
                torch.zeros(T * K, dtype=torch.int32), torch.zeros(T, K, dtype=torch.int32, device="meta")):
        with pytest.raises(ValueError, match="ids"):
            qlora.forward(layer, *ads, x, bad, gates)
    assert not calls
