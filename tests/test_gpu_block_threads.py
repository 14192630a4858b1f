"""The delta rule and the norms between blocks called from several Python
threads."""
import ctypes
import subprocess
import threading
import time

import pytest
import torch

import mamba_ssd_scan_06_amd as ssd
import test_gpu_gated_delta as delta
import test_gpu_residual_norm as norms

pytestmark = pytest.mark.gpu


def block_inputs(seed, T):
    d = delta.inputs(seed, 2, T, 4, 64, 64, 2)
    n = norms.inputs(seed + 100, (2, T, 256), "bf16", "f32", True, "token", "silu", True)
    return d, n


def block_run(d, n):
    return [*ssd.ssd_gated_delta_fwd(**d, qk_l2norm=True), *ssd.ssd_residual_norm_fwd(**n)]


@pytest.fixture
def slow_library(tmp_path):
    """The short way bound to entry points that wait 0.3 s on the host and
    enqueue nothing (a launch into a full queue takes as long)."""
    src, out = tmp_path / "slow.c", tmp_path / "libslow.so"
    src.write_text("#include <unistd.h>\nint slow(void) { usleep(300000); return 0; }\n")
    subprocess.run(["gcc", "-O1", "-shared", "-fPIC", str(src), "-o", str(out)], check=True)
    lib = ssd._load()
    address = lambda f: ctypes.cast(f, ctypes.c_void_p).value
    real = [address(f) for f in (lib.ssd_gated_delta_fwd, lib.ssd_gated_delta_workspace_bytes, lib.ssd_residual_norm_fwd)]
    slow = address(ctypes.CDLL(str(out)).slow)
    ssd._fast.bind_blocks(slow, real[1], slow)
    yield
    ssd._fast.bind_blocks(*real)


def test_other_threads_run_while_a_call_waits(slow_library):
    d, n = block_inputs(120, 45)
    calls = {"delta": lambda: ssd.ssd_gated_delta_fwd(**d), "norms": lambda: ssd.ssd_residual_norm_fwd(**n)}
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


@pytest.mark.parametrize("T", [1, 9, 90, 1500])
def test_threads_on_streams_of_their_own(T):
    ins = [block_inputs(121 + k, T) for k in range(3)]
    want = [[t.clone() for t in block_run(*i)] for i in ins]
    torch.cuda.synchronize()
    got = [[] for _ in ins]
    failed = []

    def work(k):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(8):
                    got[k].append(block_run(*ins[k]))
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
