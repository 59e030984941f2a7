"""Inputs, calls and bounds that the tests of tv_prefill and tv_decode share."""
from __future__ import annotations

import numpy as np

import oracle
import workloads


class Rows:
    """Rows of q, k, v and their decays on the device, and their values on the host.

    fused: q, k, v are views into one projection of every row.  gates: "token" (g per row),
    "head" (one per head: stride 0)."""

    def __init__(self, rng, lens, H, dk, dv, *, f32=False, diag=False, fused=False, gates="token",
                 decay=0.5, extra=0):
        import torch
        self.lens, self.H, self.dk, self.dv, self.f32, self.diag = lens, H, dk, dv, f32, diag
        self.B, self.R = len(lens), int(sum(lens)) + extra
        self.offsets = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        widths = dict(q=dk, k=dk, v=dv)
        self.host, parts = {}, {}
        for name, w in widths.items():
            x = (rng.normal(size=(self.R, H * w)) / np.sqrt(w)).astype(np.float32)
            if not f32:
                bits = workloads.f32_to_bf16_bits(x)
                x = workloads.bf16_bits_to_f32(bits)
            self.host[name] = x.reshape(self.R, H, w).astype(np.float64)
            parts[name] = torch.from_numpy(x).to("cuda", torch.float32 if f32 else torch.bfloat16)
        if fused:
            cuts = [H * w for w in widths.values()]
            both = torch.cat([parts[n] for n in widths], 1)
            parts = dict(zip(widths, both.split(cuts, 1)))
        self.dev = parts
        self.stride = {n: (x.stride(0) if self.R > 1 else sum(H * w for w in widths.values())
                           if fused else H * widths[n]) for n, x in parts.items()}
        shape = (H, dk) if diag else (H,)
        n = 1 if gates == "head" else self.R
        g = -decay * rng.exponential(size=(n,) + shape).astype(np.float32)
        self.g = torch.from_numpy(g).cuda()
        self.g_stride = 0 if gates == "head" else int(np.prod(shape))
        self.host["g"] = np.broadcast_to(g, (self.R,) + shape).astype(np.float64)

    def state(self, rng):
        import torch
        x = rng.normal(size=(self.B, self.H, self.dk, self.dv)).astype(np.float32)
        return torch.from_numpy(x).cuda(), x.astype(np.float64)

    def reference(self, H0=None):
        h = self.host
        return oracle.prefill(self.offsets, h["q"], h["k"], h["v"], h["g"], H0, self.diag)

    def magnitude(self, H0=None):
        """What the outputs and states would be with every product positive: what rounding
        errors are relative to."""
        h = {n: np.abs(x) if n != "g" else x for n, x in self.host.items()}
        return oracle.prefill(self.offsets, h["q"], h["k"], h["v"], h["g"],
                              None if H0 is None else np.abs(H0), self.diag)

    def tensor_cores(self):
        return not self.f32 and not self.diag and self.dk in (64, 128) and self.dv in (64, 128)

    def prefill(self, H0=None, out32=True, max_rows=None, workspace=True, H_new=None, stream=None,
                out=None, status=None, ws=None):
        import torch
        import tree_speculative_verify_tv_gb300 as tv
        dt = tv.TV_F32 if self.f32 else tv.TV_BF16
        decay = tv.TV_DECAY_DIAG if self.diag else tv.TV_DECAY_SCALAR
        if out is None:
            out = torch.full((self.R, self.H, self.dv), float("nan"), device="cuda",
                             dtype=torch.float32 if out32 else torch.bfloat16)
        if H_new is None:
            H_new = torch.full((self.B, self.H, self.dk, self.dv), float("nan"), device="cuda")
        if status is None:
            status = torch.zeros(1, dtype=torch.int32, device="cuda")
        max_rows = max_rows or max(1, max(self.lens))
        need = tv.tv_prefill_workspace_bytes(self.B, self.R, max_rows, self.H, self.dk, self.dv,
                                             decay, dt) if workspace is True else int(workspace)
        if ws is None and need:
            ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
        d = self.dev
        tv.tv_prefill(self.B, self.R, max_rows, self.H, self.dk, self.dv, decay, dt,
                      torch.from_numpy(self.offsets).cuda(), H0, d["q"], self.stride["q"], d["k"],
                      self.stride["k"], d["v"], self.stride["v"], self.g, self.g_stride,
                      tv.TV_F32 if out32 else tv.TV_BF16, out, H_new, ws, need, status,
                      stream=stream)
        return out, H_new, status

    def bounds(self, out32):
        """Relative (to the value) and absolute (to the magnitude) error of the outputs, and the
        absolute one of the states, from the arithmetic.

        Row by row: a row's update rounds twice (2^-24 each), the factor's pair adds 2^-24, the
        read-out sums dk products: 3 rows + dk roundings at most.
        Tensor cores: per chunk of 64 rows the state rounds twice and takes sums whose 64 / 16
        accumulations per part may each be off a whole unit (2^-23), three parts; weights carry
        two exponentials (2^-22 each), parts 2^-16 (two, bf16 outputs) or 2^-23 (three); q . k
        and q . H accumulate dk / 16 times."""
        eps, rows = 2.0 ** -24, max(self.lens + [1])
        if self.tensor_cores():
            chunks = -(-rows // 64)
            state = chunks * (4 + 24) + 8
            part = 2.0 ** -23 if out32 else 2.0 ** -15
            out = (state + 8 + 6 * self.dk // 16 + 24) * eps + 2 * part
        else:
            state = 3 * rows + 4
            out = (state + self.dk + 8) * eps
        return (eps if out32 else 2.0 ** -8), out, state * eps

    def check(self, got, H0=None, out32=True):
        import torch
        out, H_new, status = got
        torch.cuda.synchronize()
        assert int(status[0]) == 0
        want, state = self.reference(H0)
        mag, smag = self.magnitude(H0)
        rel, absolute, sabs = self.bounds(out32)
        n = int(self.offsets[-1])
        out = out[:n].float().cpu().numpy().astype(np.float64)
        H_new = H_new.cpu().numpy().astype(np.float64)
        tiny = 1e-30
        bad = np.abs(out - want[:n]) > rel * np.abs(want[:n]) + absolute * mag[:n] + tiny
        assert not (bad | ~np.isfinite(out)).any(), (
            "outputs", np.argwhere(bad | ~np.isfinite(out))[:5].tolist(),
            float(np.nanmax(np.abs(out - want[:n]) / (mag[:n] + tiny))))
        bad = np.abs(H_new - state) > sabs * smag + tiny
        assert not (bad | ~np.isfinite(H_new)).any(), (
            "states", np.argwhere(bad | ~np.isfinite(H_new))[:5].tolist(),
            float(np.nanmax(np.abs(H_new - state) / (smag + tiny))))
