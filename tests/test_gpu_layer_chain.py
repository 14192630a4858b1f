"""The operators used together, as a layer and a verify loop use them: the
projection's rows through convolution, scan and gated norm, prompt first and
then steps that carry both states; and a verify step whose accepted index goes
from ssd_verify_drafts into the states of convolution and scan on the device."""
import numpy as np
import pytest
import torch

import layer_refs as ref
import mamba_ssd_scan_06_amd as ssd
import oracle
from test_gpu_layer_ops import f64, gen, rnd, scan_inputs, verify_inputs

pytestmark = pytest.mark.gpu


class Layer:
    """One SSD layer between its projections: rows [z | x | B | C | dt] in,
    normed [b,T,H*P] out; the states are updated in place."""

    def __init__(self, g, H=8, P=64, N=64, G=2):
        self.H, self.P, self.N, self.G = H, P, N, G
        self.d, self.bc = H * P, G * N
        ch = self.d + 2 * self.bc
        self.w, self.bias = rnd(g, (ch, 4), scale=0.5), rnd(g, (ch,), scale=0.1)
        self.A = -(torch.rand(H, generator=g) * 4 + 0.5).cuda()
        self.D, self.dt_bias = rnd(g, (H,)), (rnd(g, (H,)) - 3.0)
        self.norm_w = 1 + rnd(g, (self.d,), scale=0.1)
        self.width = 2 * self.d + 2 * self.bc + H

    def states(self, b):
        return (torch.zeros(b, 3, self.d + 2 * self.bc, dtype=torch.bfloat16, device="cuda"),
                torch.zeros(b, self.H, self.P, self.N, device="cuda"))

    def parts(self, rows):
        return rows.split([self.d, self.d + 2 * self.bc, self.H], dim=2)

    def dt(self, raw):
        return torch.nn.functional.softplus(raw.float() + self.dt_bias).contiguous()

    def __call__(self, rows, conv, state, idx=None, keep=True):
        """With idx the states after that token come back too; keep writes the
        states after the last token over the given ones."""
        z, xbc, raw = self.parts(rows)
        b, T = rows.shape[:2]
        (x, B, C), _, conv_at = ssd.ssd_causal_conv_fwd(
            xbc, self.w, self.bias, conv, idx, split=[self.d, self.bc, self.bc],
            final_state=conv if keep else None, return_final_state=keep)
        y, _, state_at = ssd.ssd_chunk_scan_fwd(
            x.view(b, T, self.H, self.P), self.dt(raw), self.A, B.view(b, T, self.G, self.N),
            C.view(b, T, self.G, self.N), self.D, state, 64, idx, final_state=state if keep else None,
            return_final_state=keep)
        o = ssd.ssd_gated_norm_fwd(y.view(b, T, self.d), z, self.norm_w, ngroups=self.G)
        return o, conv_at, state_at

    def oracle(self, rows):
        z, xbc, raw = self.parts(rows)
        b, T = rows.shape[:2]
        o, _, _, _ = ref.conv(f64(xbc), f64(self.w), f64(self.bias), None, None, True, "bf16")
        # The layer rounds the convolution's outputs to bf16 (the scan's input type).
        o = f64(torch.from_numpy(o).to(torch.bfloat16))
        f = lambda a: np.ascontiguousarray(a, np.float32)
        y, fin, _, _ = oracle.ssd_forward(
            f(o[..., :self.d]).reshape(b, T, self.H, self.P), f(f64(self.dt(raw))), f(f64(self.A)),
            f(o[..., self.d:self.d + self.bc]).reshape(b, T, self.G, self.N),
            f(o[..., self.d + self.bc:]).reshape(b, T, self.G, self.N), f(f64(self.D)), None, None)
        n, _ = ref.gated_norm(y.reshape(b * T, self.d), f64(z).reshape(b * T, self.d), f64(self.norm_w), self.G, 1e-5,
                              False, "bf16")
        return n.reshape(b, T, self.d), fin


def near(got, want, tol=2e-2):
    got = f64(got)
    e = np.abs(got - want).max() / np.abs(want).max()
    print(f"  max rel err {e:.3e}", flush=True)
    assert np.isfinite(got).all() and e <= tol, e


# The scan's bound for bf16 (2e-2 normwise) holds for the chain: the inputs it
# sees are rounded to bf16 once more (2^-8), as is the norm's output.
def test_prompt_then_steps():
    g = gen(81)
    layer = Layer(g)
    b, T, steps = 3, 77, 5
    rows = rnd(g, (b, T + steps, layer.width), "bf16")
    want, fin = layer.oracle(rows)
    conv, state = layer.states(b)
    outs = [layer(rows[:, :T], conv, state)[0]]
    for t in range(T, T + steps):
        outs.append(layer(rows[:, t:t + 1], conv, state)[0])
    torch.cuda.synchronize()
    near(torch.cat(outs, 1), want)
    near(state, fin)
    assert torch.equal(conv, layer.parts(rows)[1][:, -3:])


def test_padded_batch_of_prompts():
    # Sequences of several lengths in one padded call: the states at each
    # one's last token are those of its own unpadded call.
    g = gen(82)
    layer = Layer(g)
    lens = [40, 1, 33]
    rows = rnd(g, (3, 40, layer.width), "bf16")
    idx = torch.tensor([n - 1 for n in lens], dtype=torch.int32, device="cuda")
    conv, state = layer.states(3)
    out, conv_at, state_at = layer(rows, conv, state, idx, keep=False)
    torch.cuda.synchronize()
    for i, n in enumerate(lens):
        want, fin = layer.oracle(rows[i:i + 1, :n])
        near(out[i:i + 1, :n], want)
        near(state_at[i:i + 1], fin)
        pad = torch.zeros(3, layer.d + 2 * layer.bc, dtype=torch.bfloat16, device="cuda")
        assert torch.equal(conv_at[i], torch.cat([pad, layer.parts(rows)[1][i, :n]])[-3:])


def test_verify_step_rolls_the_states_back_on_the_device():
    g = gen(83)
    layer = Layer(g)
    b, T, K = 4, 30, 5
    rows = rnd(g, (b, T + K + 1, layer.width), "bf16")
    conv, state = layer.states(b)
    layer(rows[:, :T], conv, state)
    # The block [last token, drafts] is judged, then committed up to the
    # accepted index with no host round trip.
    block = rows[:, T:]
    out, _, _ = layer(block, conv, state, keep=False)
    p, tok, u, q = verify_inputs(84, b, K, 2000, near=1.0)
    n, nxt, tokens = ssd.ssd_verify_drafts(p, tok, u, q)
    _, conv_at, state_at = layer(block, conv, state, n, keep=False)
    torch.cuda.synchronize()
    wn, wnext, wtok = ref.verify(f64(p), tok.cpu().numpy(), f64(u), f64(q))
    assert np.array_equal(n.cpu().numpy(), wn) and np.array_equal(tokens.cpu().numpy(), wtok)
    assert len(set(wn.tolist())) > 1                     # several lengths are accepted
    for i in range(b):
        upto = T + int(wn[i]) + 1
        want, fin = layer.oracle(rows[i:i + 1, :upto])
        near(out[i:i + 1, :int(wn[i]) + 1], want[:, T:])
        near(state_at[i:i + 1], fin)
        assert torch.equal(conv_at[i], layer.parts(rows)[1][i, upto - 3:upto])


@pytest.mark.parametrize("T", [9, 600])
def test_selective_layer_prompt_then_steps(T):
    # The layer with one decay per channel and state index: convolution on a
    # slice of the projection's rows [x | z], scan with that z as its gate.
    g = gen(85)
    b, Dm, N, steps = 2, 128, 16, 3
    total = T + steps
    s = scan_inputs(g, b, total, Dm, N, 1, "bf16", True, False, True, False, 0)
    xz = rnd(g, (b, total, 2 * Dm), "bf16")
    w, bias = rnd(g, (Dm, 4), scale=0.5), rnd(g, (Dm,), scale=0.1)
    conv = torch.zeros(b, 3, Dm, dtype=torch.bfloat16, device="cuda")
    state = torch.zeros(b, Dm, N, device="cuda")
    ys = []
    for lo, hi in [(0, T)] + [(t, t + 1) for t in range(T, total)]:
        x, z = xz[:, lo:hi].split([Dm, Dm], dim=2)
        u, _, _ = ssd.ssd_causal_conv_fwd(x, w, bias, conv, final_state=conv)
        y, _, _ = ssd.ssd_selective_scan_fwd(u, s["delta"][:, lo:hi], s["A"], s["B"][:, lo:hi], s["C"][:, lo:hi],
                                             s["D"], z, s["bias"], state, delta_softplus=True, final_state=state)
        ys.append(y)
    torch.cuda.synchronize()
    u, _, _, _ = ref.conv(f64(xz[..., :Dm]), f64(w), f64(bias), None, None, True, "bf16")
    u = f64(torch.from_numpy(u).to(torch.bfloat16))
    wy, _, wf, _, _, _ = ref.selective_scan(u, f64(s["delta"]), f64(s["A"]), f64(s["B"]), f64(s["C"]), f64(s["D"]),
                                            f64(xz[..., Dm:]), f64(s["bias"]), True, None, None, "bf16")
    near(torch.cat(ys, 1), wy)
    near(state, wf)
