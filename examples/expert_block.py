"""One block of a voxel transformer with experts, on the library's rows: attention with normed and rotated
heads, then a feed-forward part of which each voxel takes its k best experts.

    h   = x + attention(R(norm(q)), R(norm(k)), v) Wo,          [q k v] = norm(x) Wqkv
    out = h + sum_j gate_j down_e(j)(gelu(up_e(j)(norm(h)))),   e, gate = the k best of norm(h) Wr

`forward` keeps what `backward` needs; `backward` returns the gradients of x and of every weight, as a
training step takes them.

    python examples/expert_block.py            (needs a GPU and the built library)
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import submanifold_sparse_convolution_submconv3d_amd as sc  # noqa: E402


def gelu(u):
    return 0.5 * u * (1.0 + torch.erf(u * 0.5 ** 0.5))


def gelu_slope(u):
    return 0.5 * (1.0 + torch.erf(u * 0.5 ** 0.5)) + u * torch.exp(-0.5 * u * u) / math.sqrt(2.0 * math.pi)


class ExpertBlock:
    """channels = heads * dim; the three axes take equal shares of a head's pairs."""

    def __init__(self, channels, heads, experts, k, hidden, dtype=torch.bfloat16, device="cuda", seed=0, eps=1e-6):
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(*shape, fan, to=dtype):
            return (torch.randn(shape, generator=g, device=device) / fan ** 0.5).to(to)

        c, d = channels, channels // heads
        self.heads, self.dim, self.k, self.eps = heads, d, k, eps
        self.gamma1, self.beta1 = torch.ones(c, device=device), torch.zeros(c, device=device)   # norms stay in fp32
        self.gamma2, self.beta2 = torch.ones(c, device=device), torch.zeros(c, device=device)
        self.w_heads = torch.ones(2 * heads, d, device=device)          # one for each query and each key head
        self.w_qkv, self.w_out = weight(c, 3 * c, fan=c), weight(c, c, fan=c)
        self.w_route = weight(c, experts, fan=c, to=torch.float32)      # and so do the scores
        self.up, self.up_bias = weight(experts, hidden, c, fan=c), torch.zeros(experts, hidden, device=device)
        self.down, self.down_bias = weight(experts, c, hidden, fan=hidden), torch.zeros(experts, c, device=device)
        self.sections = (d // 2 // 3,) * 3
        self.freqs = sc.rotary_freqs(self.sections, device=device)

    def forward(self, coords, x, batch):
        """coords int32 [N,4] grouped by batch entry, x [N,C] -> (out, what backward needs)."""
        n, h, d = x.shape[0], self.heads, self.dim
        turn = (self.w_heads, coords[:, 1:], self.freqs, self.sections)
        offsets = sc.batch_offsets(coords, batch)
        n1, stats1 = sc.submconv_layer_norm(x, self.gamma1, self.beta1, eps=self.eps, return_stats=True)
        qkv = (n1 @ self.w_qkv).view(n, 3 * h, d)
        qk, rstd = sc.submconv_head_norm_rotary(qkv[:, :2 * h], *turn, eps=self.eps, return_rstd=True)
        att, lse = sc.submconv_attention(qk[:, :h], qk[:, h:], qkv[:, 2 * h:], offsets, return_lse=True)
        mid = x + att.view(n, h * d) @ self.w_out
        n2, stats2 = sc.submconv_layer_norm(mid, self.gamma2, self.beta2, eps=self.eps, return_stats=True)
        logits = n2.float() @ self.w_route
        r = sc.submconv_route(logits, self.k)
        u = sc.submconv_grouped_linear(n2, self.up, r.offsets, bias=self.up_bias, rows=r.rows)
        a = gelu(u.float()).to(u.dtype)
        y = sc.submconv_grouped_linear(a, self.down, r.offsets, bias=self.down_bias)
        out = mid + sc.submconv_combine(y, r.slots, r.gates)
        return out, (turn, offsets, x, n1, stats1, qkv, qk, rstd, att, lse, mid, n2, stats2, logits, r, u, a, y)

    def backward(self, grad, saved):
        """Gradient of out -> {"x": of the input, and of each weight by its name}."""
        turn, offsets, x, n1, stats1, qkv, qk, rstd, att, lse, mid, n2, stats2, logits, r, u, a, y = saved
        n, h, d = x.shape[0], self.heads, self.dim
        out = {}
        dy, dgates = sc.submconv_combine_backward(grad, y, r.slots, r.rows, r.gates)
        da, out["down"], out["down_bias"] = sc.submconv_grouped_linear_backward(dy, a, self.down, r.offsets, need_bias=True)
        du = (da.float() * gelu_slope(u.float())).to(u.dtype)
        dp, out["up"], out["up_bias"] = sc.submconv_grouped_linear_backward(du, n2, self.up, r.offsets, rows=r.rows, need_bias=True)
        dlogits = sc.submconv_route_backward(dgates, logits, r.experts, r.gates)
        out["w_route"] = n2.float().t() @ dlogits
        dn2 = sc.submconv_combine(dp, r.slots) + (dlogits @ self.w_route.t()).to(x.dtype)   # the pairs' rows, and the router's
        dmid, out["gamma2"], out["beta2"] = sc.submconv_layer_norm_backward(dn2, mid, stats2, self.gamma2)
        dmid += grad
        datt = (dmid @ self.w_out.t()).view(n, h, d)
        out["w_out"] = att.view(n, h * d).t() @ dmid
        dqkv = torch.empty_like(qkv)
        dqk = dqkv[:, :2 * h]
        sc.submconv_attention_backward(datt, qk[:, :h], qk[:, h:], qkv[:, 2 * h:], att, lse, offsets, dq=dqk[:, :h], dk=dqk[:, h:],
                                       dv=dqkv[:, 2 * h:])
        _, out["w_heads"] = sc.submconv_head_norm_rotary_backward(dqk, qkv[:, :2 * h], rstd, *turn, dx=dqk)   # in place
        flat = dqkv.view(n, 3 * h * d)
        out["w_qkv"] = n1.t() @ flat
        dx, out["gamma1"], out["beta1"] = sc.submconv_layer_norm_backward(flat @ self.w_qkv.t(), x, stats1, self.gamma1)
        out["x"] = dmid + dx
        return out


def main():
    import synth
    w, coords = synth.workload(2)
    coords = torch.from_numpy(coords).cuda()
    block = ExpertBlock(256, 4, experts=8, k=2, hidden=1024)
    x = torch.randn(coords.shape[0], 256, device="cuda").to(torch.bfloat16)
    for _ in range(2):
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        out, saved = block.forward(coords, x, w.batch)
        grads = block.backward(torch.randn_like(out), saved)
        end.record()
        torch.cuda.synchronize()
    used = saved[-4].offsets.diff().tolist()
    print("%d voxels, 256 channels, 2 of 8 experts: forward and backward %.2f ms, |out| %.3f, |dx| %.3f, rows of the experts %s"
          % (coords.shape[0], start.elapsed_time(end), out.float().std(), grads["x"].float().std(), used))


if __name__ == "__main__":
    main()
