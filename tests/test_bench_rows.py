"""The bench's prefill rows on CPU, with a fake of the library: the GEMM that loads by TMA
multicast runs in calls of one GPU alone."""
import types

import pytest
import torch

import bench


class FakeQ8:
    def __init__(self):
        self.calls = []

    def q8_quantize_rows(self, w):
        return w, w

    def q8_gemm(self, *a):
        self.calls.append("gemm")

    def q8_gemm_w8a8(self, *a, **kw):
        self.calls.append("w8a8")

    def lib(self):
        return types.SimpleNamespace(q8_gemm_w8a8_workspace_size=lambda *a: 256)

    def workspace(self, n, dev):
        return torch.zeros(n, dtype=torch.uint8)


@pytest.mark.parametrize("world", [1, 2, 8])
def test_the_multicast_gemm_runs_on_one_gpu_alone(monkeypatch, world):
    monkeypatch.setattr(bench.synth, "SWEEP_SHAPES", [(64, 32), (32, 64)])
    monkeypatch.setattr(bench.synth, "PREFILL_M", 40)
    q8 = FakeQ8()

    def timed(fns, reps=20):
        for f in fns:
            f()
        return 1e-3
    rows = bench.prefill_rows(torch, q8, torch.device("cpu"), timed, [(1e-3, 1e-3)], world)
    assert q8.calls == (["gemm", "w8a8"] * 2 if world == 1 else ["w8a8"] * 2)
    assert sorted(n.split("_")[1] for n in rows) == sorted(q8.calls)


def test_profile_cases_are_for_one_gpu(monkeypatch):
    monkeypatch.setenv("WORLD_SIZE", "2")
    monkeypatch.setattr("sys.argv", ["bench.py", "--profile", "prefill"])
    with pytest.raises(SystemExit) as e:
        bench.main()
    assert e.value.code == 2
