"""The decode-step kernels when a wait runs out, without a fault.

MOE_TEST_STALL_GROUP gives one of a kernel's waits a target that nothing reaches
and MOE_TEST_WAIT_LIMIT_US shortens the limit.  The launch then has to end by
itself, report MOE_STATUS_TIMEOUT and write nothing outside its buffers; the
next call on the same workspace, cleared, gives the bits of a run before it.
"""
import time

import pytest
import torch

import routed_expert_ffn_renorm_b200 as moe
from routed_expert_ffn_renorm_b200 import workloads as W

from parity_util import lib_config, weights_of
from test_gpu_few import FORMS, cfg_
from test_gpu_linear import make

pytestmark = pytest.mark.gpu


def guarded(n, fill):
    """n bytes of `fill` with 1 MB of 0x5A behind them."""
    buf = torch.full((n + (1 << 20),), 0x5A, dtype=torch.uint8, device="cuda")
    buf[:n] = fill
    return buf[:n], buf[n:]


class Few:
    """One call of the few-token layer whose scratch holds anything and whose buffers are guarded."""

    def __init__(self, kw, fmt):
        self.cfg = cfg_(H=512, E=24, I=256, k=4, **kw)
        self.inp = W.make_inputs(self.cfg, device="cuda", seed=31, router=True, gate_std=0.5)
        self.c, w = lib_config(self.cfg), weights_of(self.inp)
        pack, self.call = FORMS[fmt]
        self.w = pack(w) if pack else w
        self.ws, self.ws_end = guarded(moe.workspace_bytes(self.c, self.cfg.T), 0xAB)
        out, self.out_end = guarded(self.cfg.T * 512 * 2, 0)
        self.out = out.view(torch.bfloat16).view(self.cfg.T, 512)

    def run(self):
        moe.status_clear(self.ws)
        self.call(self.c, self.inp.x, None, self.w, self.out, self.ws)
        status = moe.status_read(self.ws)
        assert (self.ws_end == 0x5A).all() and (self.out_end == 0x5A).all()
        return status, self.out.clone()


FEW = [(dict(T=7, Is=128), 0), (dict(T=16, Is=256, budget=5), 2), (dict(T=1, Is=128), 0), (dict(T=9, budget=6), 0)]


@pytest.mark.parametrize("kw,stall", FEW, ids=lambda v: str(v) if isinstance(v, int) else "_".join(
    f"{a}{b}" for a, b in v.items()))
@pytest.mark.parametrize("fmt", ["bf16", "nvfp4"])
def test_few_routing_wait_runs_out(kw, stall, fmt, monkeypatch):
    job = Few(kw, fmt)
    status, want = job.run()
    assert status == 0
    monkeypatch.setenv("MOE_TEST_WAIT_LIMIT_US", "1000")
    monkeypatch.setenv("MOE_TEST_STALL_GROUP", str(stall))
    status, _ = job.run()
    assert status == moe.MOE_STATUS_TIMEOUT
    monkeypatch.undo()
    status, got = job.run()
    assert status == 0 and torch.equal(got, want)


@pytest.mark.parametrize("kw", [dict(T=7, Is=128), dict(T=16), dict(T=1, Is=128)],
                         ids=lambda kw: "_".join(f"{a}{b}" for a, b in kw.items()))
@pytest.mark.parametrize("stall", [0, 1])
@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
def test_few_launch_ends_soon(kw, stall, fmt, monkeypatch):
    """Every role stops once one has given up: no wait for a copy that nobody issued lasts its 4 s."""
    job = Few(kw, fmt)
    status, want = job.run()
    assert status == 0
    monkeypatch.setenv("MOE_TEST_WAIT_LIMIT_US", "1000")
    monkeypatch.setenv("MOE_TEST_STALL_GROUP", str(stall))
    t0 = time.perf_counter()
    status, _ = job.run()
    dt = time.perf_counter() - t0
    assert status == moe.MOE_STATUS_TIMEOUT
    assert dt < 2.0, f"the aborted launch took {dt:.2f} s"
    monkeypatch.undo()
    status, got = job.run()
    assert status == 0 and torch.equal(got, want)


@pytest.mark.parametrize("env", [{"MOE_TEST_WAIT_LIMIT_US": "0"}, {"MOE_TEST_STALL_GROUP": "3"}])
def test_few_hooks_reject_bad_values(env, monkeypatch):
    job = Few(dict(T=2), "bf16")
    for k, v in env.items():
        monkeypatch.setenv(k, v)
    with pytest.raises(moe.MoEError):
        job.run()


LINEAR = [(7, 300, 1040), (7, 19200, 1040), (16, 4096, 1024), (64, 500, 8200), (70, 384, 5128), (224, 5120, 4096),
          (280, 9608, 72), (300, 9480, 2048)]


@pytest.mark.parametrize("T,N,K", LINEAR)
@pytest.mark.parametrize("stall", [0, 3])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_linear_wait_runs_out(T, N, K, stall, dtype, monkeypatch):
    """A ring slot that never fills, in single CTAs and pairs, whole tiles (staged or not) and shared ones."""
    x, w, b, r = make(T, N, K, True, True, 32)
    size = 2 if dtype == torch.bfloat16 else 4
    ws, ws_end = guarded(moe.linear_workspace_bytes(T, N, K), 0xAB)
    out, out_end = guarded(T * N * size, 0)
    out = out.view(dtype).view(T, N)

    def run():
        moe.status_clear(ws)
        moe.moe_linear(x, w, out, ws, bias=b, activation="gelu", residual=r)
        status = moe.status_read(ws)
        assert (ws_end == 0x5A).all() and (out_end == 0x5A).all()
        return status, out.clone()

    status, want = run()
    assert status == 0
    monkeypatch.setenv("MOE_TEST_WAIT_LIMIT_US", "1000")
    monkeypatch.setenv("MOE_TEST_STALL_GROUP", str(stall))
    t0 = time.perf_counter()
    status, _ = run()
    dt = time.perf_counter() - t0
    assert status == (moe.MOE_STATUS_TIMEOUT if stall < workers(T, N, K, dtype) else 0)
    assert dt < 2.0, f"the aborted launch took {dt:.2f} s"
    monkeypatch.undo()
    status, got = run()
    assert status == 0 and torch.equal(got, want)


def workers(T, N, K, dtype):
    """At least 4 CTAs or pairs, if the map has 4 row tiles or K slices to share."""
    return 4 if (N + 255) // 256 >= 4 or K >= 2048 else 1


def test_linear_hooks_reject_bad_values(monkeypatch):
    x, w, _, _ = make(2, 16, 16, False, False)
    ws = torch.zeros(moe.linear_workspace_bytes(2, 16, 16), dtype=torch.uint8, device="cuda")
    monkeypatch.setenv("MOE_TEST_STALL_GROUP", "161")
    with pytest.raises(moe.MoEError):
        moe.moe_linear(x, w, torch.empty(2, 16, device="cuda"), ws)
