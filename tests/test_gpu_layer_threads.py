"""The operators around the scan called from several Python threads."""
import ctypes
import subprocess
import threading
import time

import pytest
import torch

import mamba_ssd_scan_06_amd as ssd
from test_gpu_layer_ops import layer_inputs, layer_run

pytestmark = pytest.mark.gpu


@pytest.fixture
def slow_library(tmp_path):
    """The short way bound to entry points that wait 0.3 s on the host and
    enqueue nothing (a launch into a full queue takes as long)."""
    src, out = tmp_path / "slow.c", tmp_path / "libslow.so"
    src.write_text("#include <unistd.h>\nint slow(void) { usleep(300000); return 0; }\n")
    subprocess.run(["gcc", "-O1", "-shared", "-fPIC", str(src), "-o", str(out)], check=True)
    lib = ssd._load()
    address = lambda f: ctypes.cast(f, ctypes.c_void_p).value
    real = [address(f) for f in (lib.ssd_causal_conv_fwd, lib.ssd_selective_scan_fwd,
                                 lib.ssd_selective_scan_workspace_bytes, lib.ssd_gated_norm_fwd, lib.ssd_verify_drafts,
                                 lib.ssd_verify_workspace_bytes)]
    slow = address(ctypes.CDLL(str(out)).slow)
    ssd._fast.bind(slow, slow, real[2], slow, slow, real[5])
    yield
    ssd._fast.bind(*real)


def test_other_threads_run_while_a_call_waits(slow_library):
    s, c, nrm, ver = layer_inputs(111, 45)
    calls = {
        "conv": lambda: ssd.ssd_causal_conv_fwd(*c),
        "scan": lambda: ssd.ssd_selective_scan_fwd(s["u"], s["delta"], s["A"], s["B"], s["C"]),
        "norm": lambda: ssd.ssd_gated_norm_fwd(*nrm),
        "verify": lambda: ssd.ssd_verify_drafts(*ver),
    }
    ticks, done = [0], threading.Event()

    def tick():
        while not done.wait(0.001):
            ticks[0] += 1

    other = threading.Thread(target=tick)
    other.start()
    try:
        for name, call in calls.items():
            before, start = ticks[0], time.monotonic()
            call()
            took, ran = time.monotonic() - start, ticks[0] - before
            print(f"\n  {name}: {ran} turns of the other thread in {took:.3f} s", flush=True)
            assert took >= 0.29, f"{name} did not take the short way"
            assert ran >= 20, f"{name} held the interpreter lock"
    finally:
        done.set()
        other.join()


@pytest.mark.parametrize("T", [1, 1200])
def test_threads_on_streams_of_their_own(T):
    ins = [layer_inputs(112 + k, T) for k in range(3)]
    want = [[t.clone() for t in layer_run(*i)] for i in ins]
    torch.cuda.synchronize()
    got = [[] for _ in ins]
    failed = []

    def work(k):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(8):
                    got[k].append(layer_run(*ins[k]))
        except Exception as e:                         # reported by the main thread
            failed.append((k, e))

    threads = [threading.Thread(target=work, args=(k,)) for k in range(len(ins))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    for k in range(len(ins)):
        for turn, outs in enumerate(got[k]):
            for i, (a, b) in enumerate(zip(outs, want[k])):
                assert torch.equal(a, b), (k, turn, i)
