"""Mamba blocks around the library's operators, served and trained.

    python examples/mamba_block.py

serve(): a batch of prompts of different lengths goes through the block packed, every request's
convolution history and scan state ending up in its cache slot; the requests then generate
token by token on the same slots.  The tokens' outputs are compared with those of the whole
sequences run as prompts.

train(): the block's forward and backward pass by the library's kernels, the matrix products by
torch; the directional derivative of the loss is compared with a difference of two forward passes.

The block:  x, z = in_proj(u);  x = silu(conv(x));  dt, B, C = x_proj(x);  y = scan(x, dt, A, B, C, D);
h = residual + scale * norm(out_proj(norm(y * silu(z))));  the next block's input is norm(h).

HeadBlock is the same with heads: one step size and decay for each head, y = linear attention of the
queries C, keys B and values x with the decays dt A; each head's output is layer normed and gated, and
layer norms stand between the blocks:  h = residual + out_proj(layernorm(y) * silu(z)).
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import selective_state_space_20_amd as sss  # noqa: E402

WIDTH, STATES = 4, 16


class Block:
    def __init__(self, model_dim, dtype, seed=0, device="cuda:0"):
        g = torch.Generator(device=device).manual_seed(seed)
        rnd = lambda *s, scale=1.0: torch.randn(*s, device=device, generator=g) * scale
        inner, rank = 2 * model_dim, max(4, model_dim // 16)
        self.model_dim, self.inner, self.rank, self.dtype = model_dim, inner, rank, dtype
        self.in_proj = rnd(model_dim, 2 * inner, scale=model_dim ** -0.5).to(dtype)
        self.x_proj = rnd(inner, rank + 2 * STATES, scale=inner ** -0.5).to(dtype)
        self.dt_proj = rnd(rank, inner, scale=rank ** -0.5).to(dtype)
        self.out_proj = rnd(inner, model_dim, scale=inner ** -0.5).to(dtype)
        self.conv_w, self.conv_b = rnd(inner, WIDTH, scale=0.5), rnd(inner, scale=0.1)
        self.A = -torch.exp(torch.rand(inner, STATES, device=device, generator=g) * 2.77)
        self.D, self.dt_bias = rnd(inner), rnd(inner, scale=0.5) - 4.0
        self.gate_w, self.post_w, self.next_w = (1 + rnd(n, scale=0.1) for n in (inner, model_dim, model_dim))
        self.scale = rnd(model_dim, scale=0.3)

    def cache(self, slots):
        dev = self.A.device
        return (torch.zeros(slots, WIDTH - 1, self.inner, dtype=self.dtype, device=dev),
                torch.zeros(slots, self.inner, STATES, device=dev))

    def _split(self, u):
        xz = u @ self.in_proj
        return xz[:, :self.inner], xz[:, self.inner:]  # halves of the same rows: taken as they lie

    def _project(self, x):
        rows = x @ self.x_proj
        dt = rows[:, :self.rank] @ self.dt_proj
        return dt, rows[:, self.rank:self.rank + STATES], rows[:, self.rank + STATES:]

    def _finish(self, y, z, residual):
        out = sss.rms_norm_gated_fwd(y, self.gate_w, z) @ self.out_proj
        return sss.rms_norm_residual_fwd(out, self.next_w, residual, post_weight=self.post_w, scale=self.scale)

    def prompts(self, u, residual, cu_seqlens, cache, slots, continued):
        """u (tokens, model_dim): the sequences one after the other."""
        x, z = self._split(u)
        x = sss.causal_conv1d_packed_fwd(x, self.conv_w, self.conv_b, cu_seqlens=cu_seqlens, conv_state=cache[0],
                                         state_indices=slots, has_initial=continued, silu=True)
        dt, B, C = self._project(x)
        y = sss.selective_scan_packed_fwd(x, dt, self.A, B, C, self.D, cu_seqlens=cu_seqlens, state=cache[1],
                                          state_indices=slots, has_initial=continued, delta_bias=self.dt_bias,
                                          delta_softplus=True)
        return self._finish(y, z, residual)

    def step(self, u, residual, cache, slots):
        """u (requests, model_dim): one token of each request."""
        x, z = self._split(u)
        x = sss.causal_conv1d_update(x, self.conv_w, self.conv_b, conv_state=cache[0], state_indices=slots, silu=True)
        dt, B, C = self._project(x)
        y = sss.selective_state_update_slots(x, dt, self.A, B, C, self.D, state=cache[1], state_indices=slots,
                                             delta_bias=self.dt_bias, delta_softplus=True)
        return self._finish(y, z, residual)

    # ------------------------------------------------------------------------- training
    def forward(self, u, residual):
        """u, residual (batch, length, model_dim) -> (out, residual_out, what backward needs)."""
        bt, length, _ = u.shape
        k = {"u": u}
        k["xz"] = u @ self.in_proj
        k["conv_in"] = k["xz"][..., :self.inner].contiguous()
        k["x"] = sss.causal_conv1d_fwd(k["conv_in"], self.conv_w, self.conv_b, silu=True)
        k["rows"] = k["x"] @ self.x_proj
        k["dt"] = k["rows"][..., :self.rank] @ self.dt_proj
        k["B"], k["C"] = (v.float().contiguous() for v in k["rows"][..., self.rank:].split(STATES, -1))
        k["y"] = sss.selective_scan_fwd(k["x"], k["dt"], self.A, k["B"], k["C"], self.D, delta_bias=self.dt_bias,
                                        delta_softplus=True, return_last=False)
        flat = lambda v: v.reshape(bt * length, v.shape[-1])
        k["z"] = flat(k["xz"])[:, self.inner:]
        k["g"], k["g_rstd"] = sss.rms_norm_gated_fwd(flat(k["y"]), self.gate_w, k["z"], return_rstd=True)
        k["o"] = k["g"] @ self.out_proj
        out, h, k["rstd"], k["rstd_post"] = sss.rms_norm_residual_fwd(
            k["o"], self.next_w, flat(residual), post_weight=self.post_w, scale=self.scale, return_rstd=True)
        k["h"] = h
        return out.view(bt, length, -1), h.view(bt, length, -1), k

    def backward(self, dout, dh, k):
        """Gradients by name for the upstream gradients of forward's two results."""
        bt, length, _ = dout.shape
        flat = lambda v: v.reshape(bt * length, v.shape[-1])
        d = {}
        r = sss.rms_norm_residual_bwd(flat(dout), flat(dh), x=k["o"], residual_out=k["h"], weight=self.next_w,
                                      rstd=k["rstd"], post_weight=self.post_w, scale=self.scale, rstd_post=k["rstd_post"])
        d["next_w"], d["post_w"], d["scale"], d["residual"] = (r[n] for n in ("dweight", "dpost_weight", "dscale", "dresidual"))
        d["out_proj"] = k["g"].t() @ r["dx"]
        dxz = torch.empty_like(k["xz"])  # the gradients of both halves go where in_proj's backward reads them
        n = sss.rms_norm_gated_bwd(r["dx"] @ self.out_proj.t(), flat(k["y"]), self.gate_w, k["z"], rstd=k["g_rstd"],
                                   dz=flat(dxz)[:, self.inner:])
        d["gate_w"] = n["dweight"]
        s = sss.selective_scan_bwd(k["x"], k["dt"], self.A, k["B"], k["C"], self.D, dy=n["dx"].view_as(k["y"]),
                                   delta_bias=self.dt_bias, delta_softplus=True, want_dh0=False)
        d["A"], d["D"], d["dt_bias"] = s["dA"], s["dD"], s["ddelta_bias"]
        ddt = s["ddelta"].to(self.dtype)
        d["dt_proj"] = flat(k["rows"])[:, :self.rank].t() @ flat(ddt)
        drows = torch.cat([ddt @ self.dt_proj.t(), s["dB"].to(self.dtype), s["dC"].to(self.dtype)], -1)
        d["x_proj"] = flat(k["x"]).t() @ flat(drows)
        c = sss.causal_conv1d_bwd(k["conv_in"], self.conv_w, self.conv_b, dout=s["dx"] + drows @ self.x_proj.t(),
                                  silu=True, dx=dxz[..., :self.inner])
        d["conv_w"], d["conv_b"] = c["dweight"], c["dbias"]
        d["in_proj"] = flat(k["u"]).t() @ flat(dxz)
        d["u"] = dxz @ self.in_proj.t()
        return d


class HeadBlock:
    def __init__(self, model_dim, dtype, seed=0, device="cuda:0", head_dim=32):
        g = torch.Generator(device=device).manual_seed(seed)
        rnd = lambda *s, scale=1.0: torch.randn(*s, device=device, generator=g) * scale
        inner = 2 * model_dim
        self.model_dim, self.inner, self.heads, self.head_dim, self.dtype = model_dim, inner, inner // head_dim, head_dim, dtype
        self.in_proj = rnd(model_dim, 2 * inner, scale=model_dim ** -0.5).to(dtype)
        self.x_proj = rnd(inner, self.heads + 2 * STATES, scale=inner ** -0.5).to(dtype)
        self.out_proj = rnd(inner, model_dim, scale=inner ** -0.5).to(dtype)
        self.conv_w, self.conv_b = rnd(inner, WIDTH, scale=0.5), rnd(inner, scale=0.1)
        self.A = -torch.exp(torch.rand(self.heads, device=device, generator=g) * 2.77)
        self.D, self.dt_bias = rnd(self.heads), rnd(self.heads, scale=0.5) - 2.0
        self.head_w, self.head_b, self.next_w, self.next_b = 1 + rnd(inner, scale=0.1), rnd(inner, scale=0.1), \
            1 + rnd(model_dim, scale=0.1), rnd(model_dim, scale=0.1)

    def cache(self, slots):
        dev = self.A.device
        return (torch.zeros(slots, WIDTH - 1, self.inner, dtype=self.dtype, device=dev),
                torch.zeros(slots, self.heads, STATES, self.head_dim, device=dev))

    def _split(self, u):
        xz = u @ self.in_proj
        return xz[:, :self.inner], xz[:, self.inner:]

    def _operands(self, x):
        """Queries, keys, values, log decays and step sizes (and the projection's rows) of x (rows, inner)."""
        rows = x @ self.x_proj
        step = torch.nn.functional.softplus(rows[:, :self.heads].float() + self.dt_bias)
        k = rows[:, self.heads:self.heads + STATES].unflatten(1, (1, STATES))  # B and C, shared by all heads
        q = rows[:, self.heads + STATES:].unflatten(1, (1, STATES))
        return q, k, x.unflatten(1, (self.heads, self.head_dim)), step * self.A, step, rows

    def _finish(self, y, z, residual):
        y = sss.layer_norm_fwd(y.flatten(1), self.head_w, self.head_b, group_size=self.head_dim)
        return sss.layer_norm_fwd((y * torch.nn.functional.silu(z)) @ self.out_proj, self.next_w, self.next_b, residual)

    def prompts(self, u, residual, cu_seqlens, cache, slots, continued):
        x, z = self._split(u)
        x = sss.causal_conv1d_packed_fwd(x, self.conv_w, self.conv_b, cu_seqlens=cu_seqlens, conv_state=cache[0],
                                         state_indices=slots, has_initial=continued, silu=True)
        q, k, v, g, step, _ = self._operands(x)
        y = sss.linear_attention_packed_fwd(q, k, v, g, cu_seqlens=cu_seqlens, beta=step, D=self.D, state=cache[1],
                                            state_indices=slots, has_initial=continued)
        return self._finish(y, z, residual)

    def step(self, u, residual, cache, slots):
        x, z = self._split(u)
        x = sss.causal_conv1d_update(x, self.conv_w, self.conv_b, conv_state=cache[0], state_indices=slots, silu=True)
        q, k, v, g, step, _ = self._operands(x)
        y = sss.linear_attention_update_slots(q, k, v, g, beta=step, D=self.D, state=cache[1], state_indices=slots)
        return self._finish(y, z, residual)

    def forward(self, u, residual):
        bt, length, _ = u.shape
        flat = lambda v: v.reshape(bt * length, v.shape[-1])
        k = {"u": u, "cu": torch.arange(bt + 1, dtype=torch.int32, device=u.device) * length}
        k["xz"] = u @ self.in_proj
        k["conv_in"] = k["xz"][..., :self.inner].contiguous()
        k["x"] = flat(sss.causal_conv1d_fwd(k["conv_in"], self.conv_w, self.conv_b, silu=True))
        k["ops"] = self._operands(k["x"])
        q, key, v, g, step, _ = k["ops"]
        k["y"] = sss.linear_attention_packed_fwd(q, key, v, g, cu_seqlens=k["cu"], beta=step, D=self.D).flatten(1)
        k["n"], *k["head_stats"] = sss.layer_norm_fwd(k["y"], self.head_w, self.head_b, group_size=self.head_dim, return_stats=True)
        k["z"] = flat(k["xz"])[:, self.inner:]
        k["gated"] = k["n"] * torch.nn.functional.silu(k["z"])
        out, h, *k["stats"] = sss.layer_norm_fwd(k["gated"] @ self.out_proj, self.next_w, self.next_b, flat(residual),
                                                 return_stats=True)
        k["h"] = h
        return out.view(bt, length, -1), h.view(bt, length, -1), k

    def backward(self, dout, dh, k):
        bt, length, _ = dout.shape
        flat = lambda v: v.reshape(bt * length, v.shape[-1])
        d = {}
        r = sss.layer_norm_bwd(flat(dout), k["h"], self.next_w, mean=k["stats"][0], rstd=k["stats"][1], bias=True,
                               dresidual_out=flat(dh))
        d["next_w"], d["next_b"], d["residual"] = r["dweight"], r["dbias"], r["dresidual"]
        d["out_proj"] = k["gated"].t() @ r["dx"]
        dgated, sg = r["dx"] @ self.out_proj.t(), torch.sigmoid(k["z"])
        dxz = torch.empty_like(k["xz"])
        flat(dxz)[:, self.inner:] = dgated * k["n"] * sg * (1 + k["z"] * (1 - sg))
        n = sss.layer_norm_bwd((dgated * k["z"] * sg).contiguous(), k["y"], self.head_w, mean=k["head_stats"][0],
                               rstd=k["head_stats"][1], bias=True, group_size=self.head_dim)
        d["head_w"], d["head_b"] = n["dweight"], n["dbias"]
        q, key, v, g, step, rows = k["ops"]
        a = sss.linear_attention_packed_bwd(q, key, v, g, dout=n["dx"].unflatten(1, (self.heads, self.head_dim)), cu_seqlens=k["cu"],
                                            beta=step, D=self.D)
        d["D"], d["A"] = a["dD"], (a["dlog_decay"] * step).sum(0)
        ddt = (a["dbeta"] + a["dlog_decay"] * self.A) * torch.sigmoid(rows[:, :self.heads].float() + self.dt_bias)
        d["dt_bias"] = ddt.sum(0)
        drows = torch.cat([ddt.to(self.dtype), a["dk"].flatten(1), a["dq"].flatten(1)], -1)
        d["x_proj"] = k["x"].t() @ drows
        c = sss.causal_conv1d_bwd(k["conv_in"], self.conv_w, self.conv_b, silu=True, dx=dxz[..., :self.inner],
                                  dout=(a["dv"].flatten(1) + drows @ self.x_proj.t()).view_as(k["conv_in"]))
        d["conv_w"], d["conv_b"] = c["dweight"], c["dbias"]
        d["in_proj"] = flat(k["u"]).t() @ flat(dxz)
        d["u"] = dxz @ self.in_proj.t()
        return d


def serve(model_dim=256, lengths=(37, 1, 130, 64), new_tokens=6, dtype=torch.float32, device="cuda:0", kind=Block):
    """The largest difference between generated and whole-prompt outputs, relative to the largest value."""
    block, n = kind(model_dim, dtype, device=device), len(lengths)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=device)
    starts = lambda ls: i32([sum(ls[:i]) for i in range(len(ls) + 1)])
    g = torch.Generator(device=device).manual_seed(1)
    whole = [torch.randn(ln + new_tokens, model_dim, device=device, generator=g).to(dtype) for ln in lengths]
    res = [torch.randn(ln + new_tokens, model_dim, device=device, generator=g) for ln in lengths]
    slots = i32(list(range(n))[::-1])

    cache = block.cache(n)
    fresh = torch.zeros(n, dtype=torch.bool, device=device)
    want, _ = block.prompts(torch.cat(whole), torch.cat(res), starts([ln + new_tokens for ln in lengths]), cache, slots, fresh)
    want = torch.stack([w[-new_tokens:] for w in want.split([ln + new_tokens for ln in lengths])], 1)

    cache = block.cache(n + 2)
    cut = [max(1, ln // 2) for ln in lengths]  # a prompt may come in pieces
    first = torch.cat([w[:c] for w, c in zip(whole, cut)]), torch.cat([r[:c] for r, c in zip(res, cut)])
    block.prompts(*first, starts(cut), cache, slots, fresh)
    rest = [ln - c for ln, c in zip(lengths, cut)]  # some are done: an empty sequence
    second = (torch.cat([w[c:ln] for w, c, ln in zip(whole, cut, lengths)]),
              torch.cat([r[c:ln] for r, c, ln in zip(res, cut, lengths)]))
    block.prompts(*second, starts(rest), cache, slots, ~fresh)
    got = [block.step(torch.stack([w[ln + i] for w, ln in zip(whole, lengths)]),
                      torch.stack([r[ln + i] for r, ln in zip(res, lengths)]), cache, slots)[0] for i in range(new_tokens)]
    got = torch.stack(got)
    return float((got.float() - want.float()).abs().max() / want.float().abs().max())


def train(model_dim=96, batch=2, length=50, device="cuda:0", kind=Block):
    """{parameter: (directional derivative by backward, by central differences)}."""
    block = kind(model_dim, torch.float32, seed=3, device=device)
    g = torch.Generator(device=device).manual_seed(4)
    rnd = lambda *s: torch.randn(*s, device=device, generator=g)
    u, residual = rnd(batch, length, model_dim), rnd(batch, length, model_dim)
    dout, dh = rnd(batch, length, model_dim), rnd(batch, length, model_dim)

    def loss():
        out, h, _ = block.forward(u, residual)
        return float((dout.double() * out.double()).sum() + (dh.double() * h.double()).sum())

    _, _, kept = block.forward(u, residual)
    grads = block.backward(dout, dh, kept)
    found = {}
    for name, grad in grads.items():
        at = {"u": u, "residual": residual}.get(name)
        at = getattr(block, name) if at is None else at
        grad = grad.reshape(at.shape)
        step = grad / grad.norm()  # along the gradient: the largest difference there is
        eps = 2e-3 * float(at.norm()) / at.numel() ** 0.5
        at += eps * step
        up = loss()
        at -= 2 * eps * step
        down = loss()
        at += eps * step
        found[name] = (float(grad.norm()), (up - down) / (2 * eps))
    return found


if __name__ == "__main__":
    for block in (Block, HeadBlock):
        for dt in (torch.float32, torch.bfloat16):
            print(f"{block.__name__} serve {dt}: generated against whole prompts, relative difference "
                  f"{serve(dtype=dt, kind=block):.2e}")
        for name, (by_backward, by_difference) in train(kind=block).items():
            print(f"{block.__name__} train {name:9s} derivative along the gradient {by_backward:.6g}, by differences "
                  f"{by_difference:.6g}")
