"""Shapes of the experts' 8-bit products for each form of the kernel on a device with `sms`
SMs: a cluster of CTAs per tile (few tiles), a CTA per tile, a pair of CTAs per tile (more
than 104 rows per expert).  Except for the cluster form's, every CTA (pair) has several
tiles, with more blocks of 128 channels than its rings have stages.

The rule, as expert_matmul_int8.cu has it: tiles of 256 outputs (128 with SwiGLU); a
cluster of 2, 4 or 8 CTAs as long as runs of 32 rows x tiles x CTAs is at most the SMs."""
import torch

FORMS = ["cluster", "cta", "pair"]


def outputs(tiles, swiglu):
    """N of so many tiles, the last of them part empty."""
    return tiles * (128 if swiglu else 256) - 37


def shape(form, swiglu, sms):
    """-> offsets (list), K, N.  K ends inside a block of 128 channels."""
    if form == "cluster":      # two runs x tiles, at least two CTAs for each
        return [0, 0, 5, 5, 13], 1040, outputs(max(1, sms // 32), swiglu)
    if form == "cta":          # 7 experts with rows, of at most 104 on average
        ends = [0, 31, 31, 32, 96, 160, 161, 290, 330]
        return ends, 528 + 16, outputs(sms * 5 // 16, swiglu)
    ends = [0, 400, 400, 657, 1300]                       # runs of 200, 129 and 215 to 256
    return ends, 784, outputs(sms * 3 // 16, swiglu)      # 7 blocks, the last of 16 channels


def inputs(form, swiglu, sms, seed, lim=40, extra=0, K=None):
    """x, x_sf, w, w_sf, offsets with `extra` rows behind the last expert's."""
    ends, k, N = shape(form, swiglu, sms)
    K = k if K is None else K
    r = torch.Generator().manual_seed(seed)
    E, M, R = len(ends) - 1, N * (2 if swiglu else 1), ends[-1] + extra

    def ints(*size):
        return torch.randint(-lim, lim + 1, size, generator=r, dtype=torch.int32).to(torch.int8)

    xs = torch.rand(R, generator=r) * 0.02 + 0.01
    ws = (torch.rand(E, M, generator=r) + 0.5) / (lim * K ** 0.5)
    return ints(R, K), xs, ints(E, M, K), ws, torch.tensor(ends, dtype=torch.int32)
