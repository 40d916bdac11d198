"""One block of a voxel transformer on the library's rows: a submanifold convolution, then
self-attention between the voxels of each batch entry.

    h   = submanifold convolution of the features
    out = h + attention(rotate(q), rotate(k), v) Wo,   [q k v] = norm(h) Wqkv

Rows are active voxels throughout: the rulebook, the rotation's positions and the batch
offsets all come from one coordinate tensor.  `backward` returns the gradients of the
attention branch (its weights and its input h), as a training step takes them.

    python examples/voxel_block.py            (needs a GPU and the built library)
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import submanifold_sparse_convolution_submconv3d_amd as sc  # noqa: E402


class VoxelBlock:
    """channels = heads * dim; the three axes take equal shares of a head's pairs."""

    def __init__(self, channels, heads, dtype=torch.bfloat16, device="cuda", seed=0, eps=1e-6):
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(*shape, fan):
            return (torch.randn(shape, generator=g, device=device) / fan ** 0.5).to(dtype)

        c, d = channels, channels // heads
        self.channels, self.heads, self.dim, self.eps = c, heads, d, eps
        self.conv = weight(c, 3, 3, 3, c, fan=27 * c)
        self.conv_bias = torch.zeros(c, device=device)
        self.gamma = torch.ones(c, device=device)            # norm parameters stay in fp32
        self.beta = torch.zeros(c, device=device)
        self.w_qkv, self.w_out = weight(c, 3 * c, fan=c), weight(c, c, fan=c)
        self.sections = (d // 2 // 3,) * 3
        self.freqs = sc.rotary_freqs(self.sections, device=device)

    def forward(self, coords, feats, rulebook, batch):
        """coords int32 [N,4] grouped by batch entry, feats [N,C] -> (out, what backward needs)."""
        n, h, d = feats.shape[0], self.heads, self.dim
        positions, offsets = coords[:, 1:], sc.batch_offsets(coords, batch)
        x = sc.submconv_forward(feats, self.conv, self.conv_bias, rulebook)
        normed, stats = sc.submconv_layer_norm(x, self.gamma, self.beta, eps=self.eps, return_stats=True)
        qkv = (normed @ self.w_qkv).view(n, 3 * h, d)
        qk = qkv[:, :2 * h]                                  # queries and keys turn together, in place
        sc.submconv_rotary(qk, positions, self.freqs, self.sections, out=qk)
        att, lse = sc.submconv_attention(qkv[:, :h], qkv[:, h:2 * h], qkv[:, 2 * h:], offsets, return_lse=True)
        out = x + att.view(n, h * d) @ self.w_out
        return out, (positions, offsets, x, normed, stats, qkv, att, lse)

    def backward(self, grad, saved):
        """Gradient of out -> {"x": of the convolution's output, and of the branch's weights}."""
        positions, offsets, x, normed, stats, qkv, att, lse = saved
        n, h, d = qkv.shape[0], self.heads, self.dim
        datt = (grad @ self.w_out.t()).view(n, h, d)
        dqkv = torch.empty_like(qkv)
        sc.submconv_attention_backward(datt, qkv[:, :h], qkv[:, h:2 * h], qkv[:, 2 * h:], att, lse, offsets,
                                       dq=dqkv[:, :h], dk=dqkv[:, h:2 * h], dv=dqkv[:, 2 * h:])
        dqk = dqkv[:, :2 * h]                                # a rotation's gradient is the inverse rotation
        sc.submconv_rotary(dqk, positions, self.freqs, self.sections, inverse=True, out=dqk)
        flat = dqkv.view(n, 3 * h * d)
        dx, dgamma, dbeta = sc.submconv_layer_norm_backward(flat @ self.w_qkv.t(), x, stats, self.gamma)
        return {"x": grad + dx, "gamma": dgamma, "beta": dbeta, "w_qkv": normed.t() @ flat,
                "w_out": att.view(n, h * d).t() @ grad}


def main():
    import synth
    w, coords = synth.workload(2)
    coords = torch.from_numpy(coords).cuda()
    block = VoxelBlock(128, 4)
    feats = torch.randn(coords.shape[0], block.channels, device="cuda").to(torch.bfloat16)
    rb = sc.submconv_build_map(coords, w.res, w.batch)
    out, saved = block.forward(coords, feats, rb, w.batch)
    grads = block.backward(torch.randn_like(out), saved)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    out, saved = block.forward(coords, feats, rb, w.batch)
    grads = block.backward(torch.randn_like(out), saved)
    end.record()
    torch.cuda.synchronize()
    print("%d voxels, %d channels, %d heads: forward and backward %.2f ms, |out| %.3f, |dgamma| %.3f"
          % (coords.shape[0], block.channels, block.heads, start.elapsed_time(end), out.float().std(), grads["gamma"].std()))


if __name__ == "__main__":
    main()
