"""The delta rule and the norms between blocks used together, as a layer and a
verify loop use them: the projection's rows through convolution, delta rule,
gated norm and the norm onto the residual stream, prompt first and then steps
that carry both states; and a verify step whose accepted index goes from
ssd_verify_drafts into both states on the device."""
import numpy as np
import pytest
import torch

import block_refs
import layer_refs
import mamba_ssd_scan_06_amd as ssd
from test_gpu_layer_ops import f64, gen, rnd, verify_inputs

pytestmark = pytest.mark.gpu


class Block:
    """Rows [z | q | k | v | gate | g | beta] and the residual stream in; the next
    block's input and the new stream out; the states are updated in place."""

    def __init__(self, g, H=4, P=64, N=64, G=2, stream="bf16"):
        self.H, self.P, self.N, self.G, self.stream = H, P, N, G, stream
        self.d, self.qk = H * P, G * N
        self.ch = 2 * self.qk + self.d
        self.w, self.bias = rnd(g, (self.ch, 4), scale=0.5), rnd(g, (self.ch,), scale=0.1)
        self.norm_w, self.post_w, self.next_w = (1 + rnd(g, (self.d,), scale=0.1) for _ in range(3))
        self.layer_scale = torch.rand(self.d, generator=g).cuda() + 0.1
        self.sizes = [self.d, self.ch, self.d, H, H]
        self.width = sum(self.sizes)

    def states(self, b):
        return (torch.zeros(b, 3, self.ch, dtype=torch.bfloat16, device="cuda"),
                torch.zeros(b, self.H, self.P, self.N, device="cuda"))

    def gates(self, g, beta):
        return (-torch.nn.functional.softplus(g.float() - 2.0)).contiguous(), torch.sigmoid(beta.float()).contiguous()

    def __call__(self, rows, stream, conv, state, idx=None, keep=True):
        z, qkv, gate, g, beta = rows.split(self.sizes, dim=2)
        b, T = rows.shape[:2]
        (q, k, v), _, conv_at = ssd.ssd_causal_conv_fwd(
            qkv, self.w, self.bias, conv, idx, split=[self.qk, self.qk, self.d],
            final_state=conv if keep else None, return_final_state=keep)
        y, _, state_at = ssd.ssd_gated_delta_fwd(
            q.view(b, T, self.G, self.N), k.view(b, T, self.G, self.N), v.view(b, T, self.H, self.P),
            *self.gates(g, beta), state, idx, qk_l2norm=True, final_state=state if keep else None,
            return_final_state=keep)
        o = ssd.ssd_gated_norm_fwd(y.view(b, T, self.d), z, self.norm_w, ngroups=self.H)
        out, stream = ssd.ssd_residual_norm_fwd(o, stream, self.next_w, post_norm=True, post_weight=self.post_w,
                                                gate=gate, gate_activation="sigmoid", layer_scale=self.layer_scale)
        return out, stream, conv_at, state_at

    def oracle(self, rows, stream):
        z, qkv, gate, g, beta = rows.split(self.sizes, dim=2)
        b, T = rows.shape[:2]
        bf16 = lambda a: f64(torch.from_numpy(np.ascontiguousarray(a)).to(torch.bfloat16))
        o, _, _, _ = layer_refs.conv(f64(qkv), f64(self.w), f64(self.bias), None, None, True, "bf16")
        # Each operator rounds its outputs to bf16, the next one's input type.
        q, k, v = np.split(bf16(o), [self.qk, 2 * self.qk], axis=2)
        g, beta = self.gates(g, beta)
        y, fin, _ = block_refs.gated_delta(q.reshape(b, T, self.G, self.N), k.reshape(b, T, self.G, self.N),
                                           v.reshape(b, T, self.H, self.P), f64(g), f64(beta), l2=True)
        flat = lambda a: a.reshape(b * T, self.d)
        n, _ = layer_refs.gated_norm(flat(bf16(y)), flat(f64(z)), f64(self.norm_w), self.H, 1e-5, False, "bf16")
        out, _, h, _ = block_refs.residual_norm(bf16(n), flat(f64(stream)), f64(self.next_w), True, f64(self.post_w),
                                                flat(f64(gate)), "sigmoid", f64(self.layer_scale), 1.0, 1.0, 1e-5,
                                                "bf16", self.stream)
        return out.reshape(b, T, self.d), h.reshape(b, T, self.d), fin


def near(name, got, want, tol=2e-2):
    got = f64(got)
    e = np.abs(got - want).max() / np.abs(want).max()
    print(f"  {name}: max rel err {e:.3e}", flush=True)
    assert np.isfinite(got).all() and e <= tol, (name, e)


# Four roundings to bf16 (2^-8 of a value each: the convolution's, the delta
# rule's and the gated norm's outputs where they fall to the other side, then the
# result's) are 1.6e-2 of the largest value at most.
@pytest.mark.parametrize("stream", ["bf16", "f32"])
def test_prompt_then_steps(stream):
    g = gen(91)
    block = Block(g, stream=stream)
    b, T, steps = 3, 77, 5
    rows, res = rnd(g, (b, T + steps, block.width), "bf16"), rnd(g, (b, T + steps, block.d), stream, 2.0)
    want, want_h, fin = block.oracle(rows, res)
    conv, state = block.states(b)
    outs = [block(rows[:, :T], res[:, :T], conv, state)[:2]]
    for t in range(T, T + steps):
        outs.append(block(rows[:, t:t + 1], res[:, t:t + 1], conv, state)[:2])
    torch.cuda.synchronize()
    near("out", torch.cat([o for o, _ in outs], 1), want)
    near("stream", torch.cat([h for _, h in outs], 1), want_h)
    near("state", state, fin)
    assert torch.equal(conv, rows.split(block.sizes, dim=2)[1][:, -3:])


def test_padded_batch_of_prompts():
    g = gen(92)
    block = Block(g)
    lens = [70, 1, 33]
    rows, res = rnd(g, (3, 70, block.width), "bf16"), rnd(g, (3, 70, block.d), "bf16")
    idx = torch.tensor([n - 1 for n in lens], dtype=torch.int32, device="cuda")
    conv, state = block.states(3)
    out, _, conv_at, state_at = block(rows, res, conv, state, idx, keep=False)
    torch.cuda.synchronize()
    for i, n in enumerate(lens):
        want, _, fin = block.oracle(rows[i:i + 1, :n], res[i:i + 1, :n])
        near("out", out[i:i + 1, :n], want)
        near("state", state_at[i:i + 1], fin)


def verify_loop(block, rows, res, T, K, p, tok, u, q, states):
    """A prompt of T tokens, a block of K drafts judged and committed up to the
    accepted index, all on the device."""
    b = rows.shape[0]
    conv, state = states
    block(rows[:, :T], res[:, :T], conv, state)
    drafts = rows[:, T:], res[:, T:]
    out, h, _, _ = block(*drafts, conv, state, keep=False)
    n, _, tokens = ssd.ssd_verify_drafts(p, tok, u, q)
    _, _, conv_at, state_at = block(*drafts, conv, state, n, keep=False)
    return out, h, n, conv_at, state_at


def test_verify_step_rolls_the_states_back_on_the_device():
    g = gen(93)
    block = Block(g)
    b, T, K = 4, 40, 5
    rows, res = rnd(g, (b, T + K + 1, block.width), "bf16"), rnd(g, (b, T + K + 1, block.d), "bf16")
    p, tok, u, q = verify_inputs(84, b, K, 2000, near=1.0)
    out, h, n, conv_at, state_at = verify_loop(block, rows, res, T, K, p, tok, u, q, block.states(b))
    torch.cuda.synchronize()
    n = n.tolist()
    assert len(set(n)) > 1                               # several lengths are accepted
    for i in range(b):
        upto = T + n[i] + 1
        want, want_h, fin = block.oracle(rows[i:i + 1, :upto], res[i:i + 1, :upto])
        near("out", out[i:i + 1, :n[i] + 1], want[:, T:])
        near("stream", h[i:i + 1, :n[i] + 1], want_h[:, T:])
        near("state", state_at[i:i + 1], fin)
        assert torch.equal(conv_at[i], rows.split(block.sizes, dim=2)[1][i, upto - 3:upto])


def test_the_loop_captured_and_replayed():
    # One graph of the whole loop on new inputs each time, with eager calls between.
    g = gen(94)
    block = Block(g)
    b, T, K = 2, 50, 4
    rows, res = rnd(g, (b, T + K + 1, block.width), "bf16"), rnd(g, (b, T + K + 1, block.d), "bf16")
    p, tok, u, q = verify_inputs(85, b, K, 500, near=1.0)
    conv, state = block.states(b)
    run = lambda: verify_loop(block, rows, res, T, K, p, tok, u, q, (conv.zero_(), state.zero_()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    for turn in range(3):
        rows.copy_(rnd(g, rows.shape, "bf16"))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        want = run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, w) for a, w in zip(got, want)), turn
