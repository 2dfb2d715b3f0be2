#!/usr/bin/env python
"""Benchmark: one step = forward, backward-data and backward-weight of every
layer of a synthetic depthwise workload, through libdwconv's C ABI.

The eight workloads (``depthwise_convolution_dwconv2d_gb300.workloads``):
  pr1        -- N=1 C=32 28x28 3x3 fp32 ("Spatial Depthwise Convolution on
                the GPU #3057", its smallest MobileNet layer);
  mobilenet  -- the PR's MobileNet layer table at batch 64, fp32;
  largek     -- 64 x 384 x {32,48,64}^2, k in {7,13,21,27,31}, fp32 and fp16
                (the MegEngine large-kernel article's setting);
  multidil   -- three 3x3 branches with dilation 1/3/5 into one concatenated
                output, bf16 (the DynamicConvolutionOperator README);
  multiplier -- 128 x 256 x 28^2, 5x5, multiplier 2, bias, bf16;
  infer      -- the MobileNet table again as an inference forward in
                channels-last layout with a fused scale / shift / ReLU6
                epilogue, fp32 and bf16 (forward only: one call per layer);
  separable  -- the MobileNet table as depthwise-separable blocks (3x3
                depthwise + 1x1, both with scale / shift / ReLU6), bf16,
                channels-last, one call per block;
  largek_infer -- the fp16 large-kernel layers (k 13..31) as an inference
                forward with a static filter: the filter cache (the
                kernel-side im2col of the MegEngine article) is built once
                before timing where the shape has a cached form.

    python bench.py [--gpus N] [--steps K] [--warmup W] [--impl gb300|reference]
                    [--workload all|pr1|mobilenet|largek|multidil|multiplier|infer|separable|largek_infer]

With no flags every workload is timed, one after another, and ONE JSON line
is printed (rank 0). Its headline (``value``, ``config``, ``roofline``,
``e2e``, ``cpu_baseline``) is the large-kernel sweep, in TFLOP/s of
valid-tap FMAs (the largest workload, and the compute-bound one);
``configs`` holds each workload's figures in short. Its whole record (ms,
GB/s, TFLOP/s, a roofline for every kernel family, every layer, an end-to-end
figure and the oracle's CPU time) goes to stderr, behind "details: ".
``value`` is measured with every input resident in HBM and L2 flushed before
every call; ``e2e`` is the same metric with pinned host buffers copied in and
results copied out inside the timed region (copies on two side streams,
overlapped with the compute of other layers). ``--impl reference`` times the
fp64 CPU oracle on a bounded sample of the headline workload instead (the
only reference that exists for this method).
"""
from __future__ import annotations

import argparse
import hashlib
import json
import os
import platform
import statistics
import subprocess
import sys
import threading
import time

ROOT = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, ROOT)

METRIC = "dwconv fwd/bwd-data/bwd-weight ms, achieved GB/s or TFLOP/s vs roofline"
FALLBACK_HBM_GBS = 6800.0
FALLBACK_BF16_TFLOPS = 1900.0
ORDER = ("pr1", "mobilenet", "largek", "multidil", "multiplier", "infer", "separable", "largek_infer")
HEADLINE = "largek"
WORKLOAD_TEXT = {
    "pr1": "PR1 layer, fp32 NCHW, N=1 C=32 H=W=28, 3x3, stride 1, pad 1, fwd+bwd_data+bwd_weight",
    "mobilenet": "MobileNet-shape sweep, fp32 NCHW, N=64, 3x3 pad 1, multiplier 1, fwd+bwd_data+bwd_weight; "
                 "layers (C,H=W,stride): (64,112,2),(128,56,1),(128,56,2),(256,28,1),(256,28,2),(512,14,1),"
                 "(512,14,2),(1024,7,2)",
    "largek": "Large-kernel depthwise, N=64 C=384, H=W in {32,48,64}, k in {7,13,21,27,31}, stride 1, pad k//2, "
              "fp32 and fp16 (fp32 accumulation), fwd+bwd_data+bwd_weight",
    "multidil": "Fused multi-dilation branches, bf16, N=2 C=64 H=W=256, 3x3 dilation 1,3,5 (pad = dilation) into "
                "one N x 3C x H x W output; fwd + bwd_data (branch sum) + bwd_weight per branch",
    "multiplier": "Depth-multiplier layer, bf16, N=128 C=256 H=W=28, m=2 (512 out channels), 5x5 pad 2, bias; "
                  "fwd+bwd_data+bwd_weight+bias grad",
    "infer": "MobileNet-shape inference forward, channels-last (NHWC in and out), N=64, 3x3 pad 1, fused "
             "per-channel scale + shift + ReLU6 (a folded batch norm), fp32 and bf16; same layer table as mobilenet",
    "separable": "MobileNet-shape depthwise-separable blocks, channels-last, bf16, N=64: 3x3 depthwise + scale + "
                 "shift + ReLU6, then 1x1 to the next layer's channels + scale + shift + ReLU6, in one call per "
                 "block; same layer table as mobilenet",
    "largek_infer": "Large-kernel inference forward with a static filter, fp16 NCHW, N=64 C=384, H=W in {32,48,64}, "
                    "k in {13,21,27,31}, stride 1, pad k//2: the filter cache (kernel-side im2col) built once before "
                    "timing where the shape has a cached form (H=W=32; H=W=64 with k<=21), the uncached forward "
                    "elsewhere",
}
# Source files holding the device code each kernel family runs (host-only
# declarations excluded): a committed DRAM traffic figure is reported only
# while these files are unchanged since its capture.
FAMILY_SOURCES = {
    "tile": ("common.cuh", "tile.cuh", "tile_plan.cuh", "tile_fit.h", "tile_cases.h", "tma.cuh",
             "tile_fwd.cu", "tile_fwd_impl.cuh", "tile_bwd2.cu", "tile_bwd2_impl.cuh", "tile_wgrad.cu",
             "tile_wgrad_impl.cuh", "tile_multi.cu", "generic.cu"),
    "plane": ("common.cuh", "plane.cu", "generic.cu"),
    "large": ("common.cuh", "tile.cuh", "large.cu", "large_entries.h", "large_common.cuh",
              "large_pair.cuh", "large_impl.cuh", "large_pwgrad.cuh", "generic.cu"),
    "ibgemm": ("common.cuh", "tma.cuh", "tma.cu", "ibgemm.cu"),
    "tcwgrad": ("common.cuh", "tma.cuh", "tma.cu", "wgrad_tc.cu", "generic.cu"),
    "generic": ("common.cuh", "generic.cu"),
    "nhwc": ("common.cuh", "nhwc.h", "nhwc.cu", "tile.cuh", "tma.cuh", "tma.cu", "vec.cuh"),
    "septc": ("common.cuh", "nhwc.h", "separable.cu", "tc.cuh", "tile.cuh", "tma.cuh", "tma.cu", "vec.cuh"),
    "ibgemm-cached": ("common.cuh", "tc.cuh", "tile.cuh", "tma.cuh", "tma.cu", "ibgemm_cache.cu"),
}


# ------------------------------------------------------------------ workload
def build_workload(name):
    from depthwise_convolution_dwconv2d_gb300 import workloads as WL
    if name == "mobilenet":
        return WL.mobilenet()
    if name == "pr1":
        return WL.pr1()
    if name == "largek":
        return WL.largek()
    if name == "multiplier":
        return WL.multiplier()
    if name == "multidil":
        return [WL.multidil()]
    if name == "infer":
        return WL.mobilenet_infer()
    if name == "separable":
        return WL.mobilenet_separable()
    if name == "largek_infer":
        return WL.largek_infer()
    raise SystemExit(f"unknown workload {name}")


def valid_taps(n_out, k, s, p, d, n_in):
    tot = 0
    for o in range(n_out):
        for a in range(k):
            i = o * s - p + a * d
            if 0 <= i < n_in:
                tot += 1
    return tot


def layer_calls(item):
    """Calls of one step for one workload item: list of (pass, bytes, fma, launches)."""
    from depthwise_convolution_dwconv2d_gb300 import workloads as WL
    if isinstance(item, WL.Multi):
        brs, ctot = item.branches()
        es = 4 if item.dtype == "f32" else 2
        xb = item.N * item.C * item.H * item.W * es
        yb = item.N * ctot * brs[0].Ho * brs[0].Wo * es
        wb = sum(L.OC * L.k * L.k * es for L in brs)
        fma = sum(L.N * L.OC * valid_taps(L.Ho, L.k, L.s, L.p, L.d, L.H) * valid_taps(L.Wo, L.k, L.s, L.p, L.d, L.W)
                  for L in brs)
        out = [("fwd", xb + wb + yb, fma, None), ("bwd_data", yb + wb + xb, fma, None)]
        for L in brs:
            out.append(("bwd_weight", xb + yb // len(brs) + L.OC * L.k * L.k * es, fma // len(brs), 2))
        return out
    L = item
    es = 4 if L.dtype == "f32" else 2
    if isinstance(L, WL.SepLayer):
        # depthwise FMAs (valid taps) + 1x1 MACs; bytes: x, y, both filters, both scale / shift pairs
        fma = L.N * L.OC * valid_taps(L.Ho, L.k, L.s, L.p, L.d, L.H) * valid_taps(L.Wo, L.k, L.s, L.p, L.d, L.W)
        fma += L.N * L.Ho * L.Wo * L.OC * L.cout
        nb = (L.N * L.C * L.H * L.W + L.N * L.cout * L.Ho * L.Wo + L.OC * (L.k * L.k + 2)
              + L.cout * (L.OC + 2)) * es
        return [("fwd", nb, fma, 1)]
    if isinstance(L, WL.InferLayer):
        fma = L.N * L.OC * valid_taps(L.Ho, L.k, L.s, L.p, L.d, L.H) * valid_taps(L.Wo, L.k, L.s, L.p, L.d, L.W)
        nb = L.N * L.C * L.H * L.W * es + L.N * L.OC * L.Ho * L.Wo * es + L.OC * (L.k * L.k + 2) * es
        return [("fwd", nb + (L.OC * es if L.bias else 0), fma, 1)]
    if isinstance(L, WL.CachedLayer):
        # bytes: x and y, plus the filter cache every call reads (the filter
        # itself where the shape has no cached form)
        from depthwise_convolution_dwconv2d_gb300 import binding as B
        fma = L.N * L.OC * valid_taps(L.Ho, L.k, L.s, L.p, L.d, L.H) * valid_taps(L.Wo, L.k, L.s, L.p, L.d, L.W)
        cache = B.dwconv2d_filter_cache_size(B.make_desc(**L.desc_kwargs()), 0)
        nb = L.N * L.C * L.H * L.W * es + L.N * L.OC * L.Ho * L.Wo * es + (cache or L.OC * L.k * L.k * es)
        return [("fwd", nb + (L.OC * es if L.bias else 0), fma, 1)]
    xb = L.N * L.C * L.H * L.W * es
    yb = L.N * L.OC * L.Ho * L.Wo * es
    wb = L.OC * L.k * L.k * es
    bb = L.OC * es if L.bias else 0
    fma = L.N * L.OC * valid_taps(L.Ho, L.k, L.s, L.p, L.d, L.H) * valid_taps(L.Wo, L.k, L.s, L.p, L.d, L.W)
    return [("fwd", xb + wb + yb + bb, fma, 1), ("bwd_data", yb + wb + xb, fma, 1),
            ("bwd_weight", xb + yb + wb + bb, fma, 2)]


def dense_fma(item):
    """One step's dense tap count of a workload item, the pages' convention:
    every output times every filter tap (N*OC*Ho*Wo*kh*kw per pass, padded
    taps included), beside the valid-tap count the roofline uses. The 1x1
    stage of a separable block has no padding: its MACs count the same in
    both."""
    from depthwise_convolution_dwconv2d_gb300 import workloads as WL
    if isinstance(item, WL.Multi):
        brs, _ = item.branches()
        per = sum(L.N * L.OC * L.Ho * L.Wo * L.k * L.k for L in brs)
        return 3 * per  # fwd, bwd_data (branch sum), bwd_weight per branch
    L = item
    per = L.N * L.OC * L.Ho * L.Wo * L.k * L.k
    if isinstance(L, WL.SepLayer):
        return per + L.N * L.Ho * L.Wo * L.OC * L.cout
    if isinstance(L, (WL.InferLayer, WL.CachedLayer)):
        return per
    return 3 * per


# ------------------------------------------------------------------ helpers
def load_peaks():
    """(HBM GB/s, its source, dense bf16 TFLOP/s burst, its source)."""
    path = os.path.join(ROOT, "MEASURED_PEAKS.json")
    hbm, hk, tc, tk = FALLBACK_HBM_GBS, "fallback", FALLBACK_BF16_TFLOPS, "fallback"
    if os.path.exists(path):
        try:
            j = json.load(open(path))
            if j.get("hbm_gbs"):
                hbm, hk = float(j["hbm_gbs"]), "measured"
            if j.get("bf16_tflops"):
                tc, tk = float(j["bf16_tflops"]), "measured"
        except Exception:
            pass
    return hbm, hk, tc, tk


def cpu_model():
    try:
        out = subprocess.run(["lscpu"], capture_output=True, text=True, timeout=10).stdout
        for ln in out.splitlines():
            if ln.strip().startswith("Model name:"):
                return ln.split(":", 1)[1].strip()
    except Exception:
        pass
    try:
        for ln in open("/proc/cpuinfo"):
            if ln.lower().startswith("model name"):
                return ln.split(":", 1)[1].strip()
    except Exception:
        pass
    return platform.processor() or platform.machine()


class ClockSampler:
    """nvidia-smi clocks and throttle reasons, sampled while a timed loop runs."""
    FIELDS = ("clocks.sm,clocks.max.sm,power.draw,clocks_event_reasons.active,"
              "clocks_event_reasons.hw_slowdown,clocks_event_reasons.hw_thermal_slowdown,"
              "clocks_event_reasons.sw_thermal_slowdown,clocks_event_reasons.sw_power_cap")

    def __init__(self, index):
        self.index = index
        self.proc = None
        self.lines = []

    def __enter__(self):
        try:
            self.proc = subprocess.Popen(
                ["nvidia-smi", "-i", str(self.index), f"--query-gpu={self.FIELDS}",
                 "--format=csv,noheader,nounits", "-lms", "100"],
                stdout=subprocess.PIPE, stderr=subprocess.DEVNULL, text=True)
            self.t = threading.Thread(target=self._read, daemon=True)
            self.t.start()
        except Exception:
            self.proc = None
        return self

    def _read(self):
        for line in self.proc.stdout:
            self.lines.append(line.strip())

    def __exit__(self, *a):
        if self.proc:
            self.proc.terminate()
            try:
                self.proc.wait(timeout=5)
            except Exception:
                self.proc.kill()


def clock_summary(lines):
    sm, mx, reasons = [], [], set()
    names = ["hw_slowdown", "hw_thermal_slowdown", "sw_thermal_slowdown", "sw_power_cap"]
    for ln in lines:
        parts = [p.strip() for p in ln.split(",")]
        if len(parts) < 8:
            continue
        try:
            sm.append(float(parts[0]))
            mx.append(float(parts[1]))
        except ValueError:
            continue
        for nm, v in zip(names, parts[4:8]):
            if v.lower() == "active":
                reasons.add(nm)
    if not sm:
        return None
    return {"sm_mhz": statistics.median(sm), "sm_max_mhz": max(mx), "samples": len(sm),
            "reasons": sorted(reasons)}


def family_digest(family):
    h = hashlib.sha256()
    d = os.path.join(ROOT, "depthwise_convolution_dwconv2d_gb300", "csrc")
    for f in FAMILY_SOURCES.get(family, ()):
        p = os.path.join(d, f)
        h.update(f.encode())
        if os.path.exists(p):
            h.update(open(p, "rb").read())
    return h.hexdigest()[:16]


def ncu_traffic(key, family):
    """Per-launch DRAM bytes of one kernel family from the committed ncu
    figures (one representative layer, scaled to the workload's batch), if
    they were taken on the family's current sources; else None."""
    path = os.path.join(ROOT, "profiles", "ncu_traffic.json")
    if not os.path.exists(path):
        return None
    try:
        e = json.load(open(path)).get("kernels", {}).get(key)
    except Exception:
        return None
    if not e or e.get("digest") != family_digest(family):
        return None
    return e


def fma_probe_tflops(dev, stream):
    """FP32 FMA peak of this GPU, measured with the library's register-only
    FMA probe (16 independent chains per thread, 8 CTAs of 256 per SM)."""
    import torch
    from depthwise_convolution_dwconv2d_gb300 import binding as B
    sink = torch.empty(152 * 8 * 256, device=dev)
    for _ in range(2):
        B.dwconv_fma_probe(152 * 8, 4096, sink, stream)
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    best = 0.0
    for _ in range(3):
        a.record(stream)
        B.dwconv_fma_probe(152 * 8, 16384, sink, stream)
        b.record(stream)
        torch.cuda.synchronize()
        best = max(best, 2 * 16 * 16384 * 152 * 8 * 256 / a.elapsed_time(b) / 1e9)
    return best


# ------------------------------------------------------------------ CPU oracle
def oracle_sample(items, budget_s):
    """Time the fp64 oracle on a bounded sample of every layer: the first n
    samples and, while even one sample takes longer than the budget, the
    first c channels. Returns (bytes/s, fma/s, seconds, description)."""
    import oracle
    from depthwise_convolution_dwconv2d_gb300 import workloads as WL
    oracle.build()

    def run(n, c_cap):
        t_total, bytes_total, fma_total = 0.0, 0, 0
        for item in items:
            C = min(item.C, c_cap)
            if isinstance(item, WL.Multi):
                brs, ctot = item.branches()
                sub = WL.Multi(N=n, C=C, H=item.H, W=item.W, dilations=item.dilations, k=item.k,
                               dtype=item.dtype, x_dist=item.x_dist, w_std=item.w_std)
                sbrs, sctot = sub.branches()
                x, gy = WL.make_x(sbrs[0]), WL.make_gy(sbrs[0], gy_channels=sctot)
                ws = [WL.make_w(L, branch=i).f64 for i, L in enumerate(sbrs)]
                cvs = [oracle.Conv(N=n, C=L.C, H=L.H, W=L.W, kh=L.k, kw=L.k, sh=L.s, sw=L.s, ph=L.p, pw=L.p,
                                   dh=L.d, dw=L.d, off=i * L.C, c_total=sctot) for i, L in enumerate(sbrs)]
                t0 = time.perf_counter()
                oracle.fwd_multi(cvs, x.f64, ws)
                oracle.bwd_data_multi(cvs, gy.f64, ws)
                for cv in cvs:
                    oracle.bwd_weight(cv, x.f64, gy.f64)
                t_total += time.perf_counter() - t0
                for _, b, f, _ in layer_calls(sub):
                    bytes_total += b
                    fma_total += f
                continue
            L = type(item)(**{**item.__dict__, "N": n, "C": C})
            inp = WL.make_inputs(L)
            cv = oracle.Conv(N=n, C=L.C, H=L.H, W=L.W, kh=L.k, kw=L.k, sh=L.s, sw=L.s, ph=L.p, pw=L.p,
                             dh=L.d, dw=L.d, m=L.m)
            b = inp.b.f64 if inp.b is not None else None
            if isinstance(L, WL.SepLayer):
                sc, sh = WL.make_scale_shift(L)
                wp, psc, psh = WL.make_pointwise(L, L.cout)
                t0 = time.perf_counter()
                oracle.separable(cv, inp.x.f64, inp.w.f64, sc.f64, sh.f64, L.act, wp.f64, psc.f64, psh.f64, L.act)
                t_total += time.perf_counter() - t0
            elif isinstance(L, WL.InferLayer):
                # the oracle is layout-free: NCHW arrays, the same function
                sc, sh = WL.make_scale_shift(L)
                t0 = time.perf_counter()
                oracle.fwd_epilogue(cv, inp.x.f64, inp.w.f64, b, sc.f64, sh.f64, L.act)
                t_total += time.perf_counter() - t0
            elif isinstance(L, WL.CachedLayer):
                t0 = time.perf_counter()
                oracle.fwd(cv, inp.x.f64, inp.w.f64, b)
                t_total += time.perf_counter() - t0
            else:
                t0 = time.perf_counter()
                oracle.fwd(cv, inp.x.f64, inp.w.f64, b)
                oracle.bwd_data(cv, inp.gy.f64, inp.w.f64)
                oracle.bwd_weight(cv, inp.x.f64, inp.gy.f64, want_b=L.bias)
                t_total += time.perf_counter() - t0
            for _, bb, f, _ in layer_calls(L):
                bytes_total += bb
                fma_total += f
        return t_total, bytes_total, fma_total

    full_c = max(i.C for i in items)
    full_n = min(i.N for i in items)
    c = min(full_c, 32)
    t, by, fm = run(1, c)
    n = 1
    if t < budget_s / 2:
        # grow the channel count first, then the batch
        scale = budget_s / max(t, 1e-3)
        if c * scale < full_c:
            c = max(c, int(c * scale) // 8 * 8)
        else:
            scale /= full_c / c
            c = full_c
            n = max(1, min(full_n, int(scale)))
        t, by, fm = run(n, c)
    passes = ("separable block (depthwise + 1x1, both epilogues)" if all(isinstance(i, WL.SepLayer) for i in items)
              else "fwd with epilogue" if all(isinstance(i, WL.InferLayer) for i in items)
              else "fwd" if all(isinstance(i, WL.CachedLayer) for i in items)
              else "fwd+bwd_data+bwd_weight")
    desc = (f"first {n} sample(s)" + ("" if c >= full_c else f" and first {c} channels") +
            f" of every layer, {passes}, one timed pass")
    return by / t, fm / t, t, desc


def cpu_baseline(name, items, budget_s, unit):
    import oracle
    bps, fps, t, desc = oracle_sample(items, budget_s)
    v = 2 * fps / 1e12 if unit == "TFLOP/s" else bps / 1e9
    return {"value": round(v, 5), "unit": unit, "cores": oracle.num_threads(), "cpu_model": cpu_model(),
            "kind": "oracle", "sample": desc, "seconds": round(t, 2),
            "GBps": round(bps / 1e9, 4), "tflops_valid": round(2 * fps / 1e12, 6)}


# ------------------------------------------------------------------ GPU arm
class _NHWC:
    """A synthetic NCHW tensor's bytes transposed to channels-last."""

    def __init__(self, t):
        import numpy as np
        self.dtype = t.dtype
        self.store = np.ascontiguousarray(t.store.transpose(0, 2, 3, 1))


class HostCache:
    """Synthetic host tensors, drawn once per (shape, dtype, stream, std) and
    pinned; layers with equal shapes share them (the device buffers are still
    one per layer)."""

    def __init__(self):
        self.t = {}

    def get(self, key, make):
        if key not in self.t:
            import torch
            import numpy as np
            st = make()
            if st.dtype == "bf16":
                h = torch.from_numpy(st.store.view(np.int16)).view(torch.bfloat16)
            else:
                h = torch.from_numpy(st.store)
            self.t[key] = h.pin_memory()
        return self.t[key]


def setup_workload(name, items, dev, stream, hc, out_host):
    """Device buffers and the call list of one step. Returns (calls, groups):
    calls = [(pass, label, family, bytes, fma, launches, fn)], groups = one
    per layer: (h2d pairs, call indices, d2h pairs)."""
    import torch
    from depthwise_convolution_dwconv2d_gb300 import binding as B, workloads as WL

    def tdt(dt):
        return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[dt]

    def host_out(t):
        key = (tuple(t.shape), t.dtype)
        if key not in out_host:
            out_host[key] = torch.empty(t.shape, dtype=t.dtype, device="cpu").pin_memory()
        return out_host[key]

    def fam(plan, dt):
        return f"{plan}:{dt}"

    calls, groups = [], []
    for item in items:
        if isinstance(item, WL.Multi):
            brs, ctot = item.branches()
            L0 = brs[0]
            xd = "uniform" if item.x_dist == "uniform" else "normal"
            xh = hc.get(("x", (item.N, item.C, item.H, item.W), item.dtype, xd), lambda: WL.make_x(L0))
            gyh = hc.get(("gy", (item.N, ctot, L0.Ho, L0.Wo), item.dtype),
                         lambda: WL.make_gy(L0, gy_channels=ctot))
            whs = [hc.get(("w", (item.C, item.k, item.k), item.dtype, i, item.w_std),
                          lambda i=i: WL.make_w(brs[i], branch=i))
                   for i in range(len(brs))]
            x, gy = xh.to(dev), gyh.to(dev)
            wdev = [h.to(dev) for h in whs]
            descs = [B.make_desc(**L.desc_kwargs(), out_c_offset=i * item.C, out_c_total=ctot)
                     for i, L in enumerate(brs)]
            y = torch.empty((item.N, ctot, L0.Ho, L0.Wo), dtype=tdt(item.dtype), device=dev)
            gx = torch.empty((item.N, item.C, item.H, item.W), dtype=tdt(item.dtype), device=dev)
            gws = [torch.empty((item.C, item.k, item.k), dtype=tdt(item.dtype), device=dev) for _ in brs]
            wss = [torch.empty(B.dwconv2d_bwd_weight_workspace_size(dd) // 4 + 4, device=dev) for dd in descs]
            cl = layer_calls(item)
            nb = len(brs)
            mplan = B.dwconv2d_multi_plan_name(descs)
            fused = mplan == "tile"
            idx0 = len(calls)
            calls.append(("fwd", item.label(), fam("multi-" + mplan, item.dtype), cl[0][1], cl[0][2],
                          1 if fused else nb,
                          lambda descs=descs, x=x, wdev=wdev, y=y: B.dwconv2d_fwd_multi(descs, x, wdev, None, y, stream)))
            calls.append(("bwd_data", item.label(), fam("multi-" + mplan, item.dtype), cl[1][1], cl[1][2], 1,
                          lambda descs=descs, gy=gy, wdev=wdev, gx=gx: B.dwconv2d_bwd_data_multi(descs, gy, wdev, gx, stream)))
            for i, dd in enumerate(descs):
                calls.append(("bwd_weight", f"{item.label()}_br{i}", fam(B.dwconv2d_plan_name(dd, 2), item.dtype),
                              cl[2 + i][1], cl[2 + i][2], 2,
                              lambda dd=dd, x=x, gy=gy, g=gws[i], ws=wss[i]: B.dwconv2d_bwd_weight(dd, x, gy, g, None, ws, None, stream)))
            h2d = [(xh, x), (gyh, gy)] + list(zip(whs, wdev))
            d2h = [(t, host_out(t)) for t in [y, gx] + gws]
            groups.append((h2d, list(range(idx0, len(calls))), d2h))
            continue
        L = item
        xd = "uniform" if L.x_dist == "uniform" else "normal"
        wstd = L.w_std if L.w_std is not None else 1.0 / L.k
        if isinstance(L, WL.SepLayer):
            xh = hc.get(("x_nhwc", (L.N, L.H, L.W, L.C), L.dtype, xd), lambda L=L: _NHWC(WL.make_x(L)))
            wh = hc.get(("w", (L.OC, L.k, L.k), L.dtype, 0, wstd), lambda L=L: WL.make_w(L))
            sch = hc.get(("scale", (L.OC,), L.dtype), lambda L=L: WL.make_scale_shift(L)[0])
            shh = hc.get(("shift", (L.OC,), L.dtype), lambda L=L: WL.make_scale_shift(L)[1])
            pws = [hc.get(("pw", i, (L.cout, L.OC), L.dtype), lambda L=L, i=i: WL.make_pointwise(L, L.cout)[i])
                   for i in range(3)]
            d = B.make_desc(**L.desc_kwargs())
            x, w, sc, sh = xh.to(dev), wh.to(dev), sch.to(dev), shh.to(dev)
            wp, psc, psh = (t.to(dev) for t in pws)
            y = torch.empty((L.N, L.Ho, L.Wo, L.cout), dtype=tdt(L.dtype), device=dev)
            cl = layer_calls(L)
            idx0 = len(calls)
            calls.append(("fwd", L.label(), fam(B.dwconv2d_separable_plan_name(d, L.cout), L.dtype), cl[0][1],
                          cl[0][2], 1,
                          lambda d=d, x=x, w=w, y=y, sc=sc, sh=sh, wp=wp, psc=psc, psh=psh, L=L:
                          B.dwconv2d_separable_nhwc(d, x, w, L.cout, wp, y, sc, sh, L.act, psc, psh, L.act, stream)))
            h2d = [(xh, x), (wh, w), (sch, sc), (shh, sh)] + list(zip(pws, (wp, psc, psh)))
            groups.append((h2d, list(range(idx0, len(calls))), [(y, host_out(y))]))
            continue
        if isinstance(L, WL.InferLayer):
            xh = hc.get(("x_nhwc", (L.N, L.H, L.W, L.C), L.dtype, xd), lambda L=L: _NHWC(WL.make_x(L)))
            wh = hc.get(("w", (L.OC, L.k, L.k), L.dtype, 0, wstd), lambda L=L: WL.make_w(L))
            sch = hc.get(("scale", (L.OC,), L.dtype), lambda L=L: WL.make_scale_shift(L)[0])
            shh = hc.get(("shift", (L.OC,), L.dtype), lambda L=L: WL.make_scale_shift(L)[1])
            d = B.make_desc(**L.desc_kwargs())
            x, w, sc, sh = xh.to(dev), wh.to(dev), sch.to(dev), shh.to(dev)
            y = torch.empty((L.N, L.Ho, L.Wo, L.OC), dtype=tdt(L.dtype), device=dev)
            cl = layer_calls(L)
            idx0 = len(calls)
            calls.append(("fwd", L.label(), fam(B.dwconv2d_plan_name(d, 4), L.dtype), cl[0][1], cl[0][2], 1,
                          lambda d=d, x=x, w=w, y=y, sc=sc, sh=sh, act=L.act:
                          B.dwconv2d_fwd_nhwc(d, x, w, None, y, sc, sh, act, stream)))
            h2d = [(xh, x), (wh, w), (sch, sc), (shh, sh)]
            groups.append((h2d, list(range(idx0, len(calls))), [(y, host_out(y))]))
            continue
        if isinstance(L, WL.CachedLayer):
            xh = hc.get(("x", (L.N, L.C, L.H, L.W), L.dtype, xd), lambda L=L: WL.make_x(L))
            wh = hc.get(("w", (L.OC, L.k, L.k), L.dtype, 0, wstd), lambda L=L: WL.make_w(L))
            d = B.make_desc(**L.desc_kwargs())
            x, w = xh.to(dev), wh.to(dev)
            y = torch.empty((L.N, L.OC, L.Ho, L.Wo), dtype=tdt(L.dtype), device=dev)
            cl = layer_calls(L)
            idx0 = len(calls)
            nbytes = B.dwconv2d_filter_cache_size(d, 0)
            if nbytes:
                # static filter: its cache is built once, outside the timed calls
                cache = torch.empty(nbytes, dtype=torch.uint8, device=dev)
                B.dwconv2d_filter_cache_build(d, 0, w, cache, None, stream)
                calls.append(("fwd", L.label(), fam("ibgemm-cached", L.dtype), cl[0][1], cl[0][2], 1,
                              lambda d=d, x=x, cache=cache, y=y: B.dwconv2d_fwd_cached(d, x, cache, None, y, None,
                                                                                      stream)))
            else:
                calls.append(("fwd", L.label(), fam(B.dwconv2d_plan_name(d, 0), L.dtype), cl[0][1], cl[0][2], 1,
                              lambda d=d, x=x, w=w, y=y: B.dwconv2d_fwd(d, x, w, None, y, stream)))
            groups.append(([(xh, x)], list(range(idx0, len(calls))), [(y, host_out(y))]))
            continue
        xh = hc.get(("x", (L.N, L.C, L.H, L.W), L.dtype, xd), lambda L=L: WL.make_x(L))
        wh = hc.get(("w", (L.OC, L.k, L.k), L.dtype, 0, wstd), lambda L=L: WL.make_w(L))
        gyh = hc.get(("gy", (L.N, L.OC, L.Ho, L.Wo), L.dtype), lambda L=L: WL.make_gy(L))
        bh = hc.get(("b", (L.OC,), L.dtype, L.b_std), lambda L=L: WL.make_b(L)) if L.bias else None
        d = B.make_desc(**L.desc_kwargs())
        x, w, gy = xh.to(dev), wh.to(dev), gyh.to(dev)
        b = bh.to(dev) if bh is not None else None
        y = torch.empty((L.N, L.OC, L.Ho, L.Wo), dtype=tdt(L.dtype), device=dev)
        gx = torch.empty((L.N, L.C, L.H, L.W), dtype=tdt(L.dtype), device=dev)
        gw = torch.empty((L.OC, L.k, L.k), dtype=tdt(L.dtype), device=dev)
        gb = torch.empty((L.OC,), dtype=tdt(L.dtype), device=dev) if L.bias else None
        ws = torch.empty(B.dwconv2d_bwd_weight_workspace_size(d) // 4 + 4, device=dev)
        cl = layer_calls(L)
        idx0 = len(calls)
        calls.append(("fwd", L.label(), fam(B.dwconv2d_plan_name(d, 0), L.dtype), cl[0][1], cl[0][2], 1,
                      lambda d=d, x=x, w=w, b=b, y=y: B.dwconv2d_fwd(d, x, w, b, y, stream)))
        calls.append(("bwd_data", L.label(), fam(B.dwconv2d_plan_name(d, 1), L.dtype), cl[1][1], cl[1][2], 1,
                      lambda d=d, gy=gy, w=w, gx=gx: B.dwconv2d_bwd_data(d, gy, w, gx, 0, stream)))
        calls.append(("bwd_weight", L.label(), fam(B.dwconv2d_plan_name(d, 2), L.dtype), cl[2][1], cl[2][2], 2,
                      lambda d=d, x=x, gy=gy, gw=gw, gb=gb, ws=ws: B.dwconv2d_bwd_weight(d, x, gy, gw, gb, ws, None, stream)))
        h2d = [(xh, x), (wh, w), (gyh, gy)] + ([(bh, b)] if b is not None else [])
        d2h = [(t, host_out(t)) for t in (y, gx, gw, gb) if t is not None]
        groups.append((h2d, list(range(idx0, len(calls))), d2h))
    return calls, groups


def roofline_of(fam_rec, bound_peaks, hbm_peak, hbm_kind, traffic_entry):
    """Roofline of one kernel family: t_roof = max(bytes / HBM peak, FLOPs /
    compute peak), frac = t_roof / t_measured; achieved in the bound's unit.
    traffic: DRAM bytes of one launch of the family's representative layer
    (ncu), beside that launch's algorithmic bytes."""
    traffic = traffic_entry.get("bytes_per_launch") if traffic_entry else None
    ms, by, fma = fam_rec["ms"], fam_rec["bytes"], fam_rec["fma"]
    comp_kind, comp_peak, comp_src = bound_peaks
    t_mem = by / (hbm_peak * 1e6)           # ms
    t_cmp = 2 * fma / (comp_peak * 1e9)     # ms
    if t_cmp > t_mem:
        ach = 2 * fma / ms / 1e9
        return {"bound": comp_kind, "achieved": round(ach, 2), "peak": round(comp_peak, 1), "unit": "TFLOP/s",
                "frac": round(ach / comp_peak, 4), "peak_source": comp_src, "work": "valid-tap FMAs x 2",
                "traffic": traffic, "hbm_frac": round(by / ms / 1e6 / hbm_peak, 4)}
    ach = by / ms / 1e6
    return {"bound": "hbm", "achieved": round(ach, 1), "peak": round(hbm_peak, 1), "unit": "GB/s",
            "frac": round(ach / hbm_peak, 4),
            "peak_source": f"{hbm_kind} ({'MEASURED_PEAKS.json hbm_gbs' if hbm_kind == 'measured' else 'profiling recipe fallback 6.8 TB/s'})",
            "work": "algorithmic bytes", "traffic": traffic,
            "compute_frac": round(2 * fma / ms / 1e9 / comp_peak, 4)}


def graph_replay_ms(calls, stream, eager_ms):
    """The step's calls captured once into a CUDA graph (no L2 flush inside)
    and replayed back to back on `stream`: ms per replay and the replay
    count, or (None, reason) if the capture failed."""
    import torch

    g = torch.cuda.CUDAGraph()
    try:
        with torch.cuda.graph(g, stream=stream):
            for c in calls:
                c[6]()
    except Exception as e:  # reported in the line, the eager timing stands
        torch.cuda.synchronize()
        return None, "capture failed: " + str(e).splitlines()[0][:200]
    reps = max(3, min(100, int(300.0 / max(eager_ms, 1e-3))))
    for _ in range(3):
        g.replay()
    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    torch.cuda.synchronize()
    e0.record(stream)
    for _ in range(reps):
        g.replay()
    e1.record(stream)
    torch.cuda.synchronize()
    ms = e0.elapsed_time(e1) / reps
    del g
    return ms, reps


def max_over_ranks(vals, dist, device="cpu"):
    """Per-rank timings (ms; None for "not measured") -> their maximum over
    all ranks, the same list on every rank. With one rank (dist None) the
    values come back unchanged."""
    if dist is None:
        return list(vals)
    import torch

    t = torch.tensor([float(v) if v is not None else 0.0 for v in vals], dtype=torch.float64, device=device)
    dist.all_reduce(t, op=dist.ReduceOp.MAX)
    return [float(x) if float(x) > 0.0 else None for x in t]


def job_throughput(world, step_units, ms, unit):
    """Whole-job throughput: every rank runs one replica of the step, so the
    units all ranks processed (world x one step's bytes or valid-tap FMAs)
    over the slowest rank's step time."""
    if unit == "TFLOP/s":
        return world * 2 * step_units / ms / 1e9
    return world * step_units / ms / 1e6


def time_workload(name, items, args, dev, stream, world, dist, peaks, fma_tflops):
    import torch
    from depthwise_convolution_dwconv2d_gb300 import binding as B
    hc, out_host = HostCache(), {}
    calls, groups = setup_workload(name, items, dev, stream, hc, out_host)
    torch.cuda.synchronize()
    step_bytes = sum(c[3] for c in calls)
    step_fma = sum(c[4] for c in calls)
    step_fma_dense = sum(dense_fma(i) for i in items)
    launches_per_step = sum(c[5] for c in calls)
    l2 = torch.cuda.get_device_properties(dev).L2_cache_size
    # L2 flush before every timed call: write a buffer of 2x L2 (evicts the
    # inputs), then read a second, clean 2x L2 buffer, so the write-back of
    # the flush's own dirty lines happens here and not inside the next timed
    # call
    nflush = max(2 * l2, 256 << 20) // 4
    flush = torch.empty(nflush, dtype=torch.float32, device=dev)
    flush_clean = torch.ones(nflush, dtype=torch.float32, device=dev)
    flush_sink = torch.empty((), dtype=torch.float32, device=dev)

    def flush_l2():
        flush.zero_()
        torch.sum(flush_clean, dim=0, out=flush_sink)

    def barrier():
        if dist is not None:
            dist.barrier()

    for _ in range(args.warmup):
        for c in calls:
            c[6]()
    torch.cuda.synchronize()

    # timed: K steps, L2 flushed before every call, per-call events
    ev = [[(torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)) for _ in calls]
          for _ in range(args.steps)]
    idx = int(os.environ.get("LOCAL_RANK", 0))
    with ClockSampler(idx) as clk:
        barrier()
        torch.cuda.synchronize()
        t_wall0 = time.perf_counter()
        for k in range(args.steps):
            for i, c in enumerate(calls):
                flush_l2()
                ev[k][i][0].record(stream)
                c[6]()
                ev[k][i][1].record(stream)
        torch.cuda.synchronize()
        barrier()
        t_wall = time.perf_counter() - t_wall0
    per_call = [[ev[k][i][0].elapsed_time(ev[k][i][1]) for i in range(len(calls))] for k in range(args.steps)]
    ms_per_step = statistics.mean(sum(r) for r in per_call)

    # end to end: per layer, inputs copied from pinned host memory on one side
    # stream, the layer's calls on the compute stream, its results copied back
    # on another side stream; layer i's copies overlap other layers' compute
    e2e_ms, h2d_bytes, d2h_bytes = None, 0, 0
    if not args.no_e2e:
        s_in, s_out = torch.cuda.Stream(device=dev), torch.cuda.Stream(device=dev)
        g_in = [torch.cuda.Event() for _ in groups]
        g_cmp = [torch.cuda.Event() for _ in groups]
        g_out = [torch.cuda.Event() for _ in groups]
        started = [False] * len(groups)

        def e2e_step():
            for gi, (h2d, idxs, d2h) in enumerate(groups):
                if started[gi]:
                    s_in.wait_event(g_cmp[gi])      # inputs are free once last step's calls ran
                with torch.cuda.stream(s_in):
                    for hsrc, ddst in h2d:
                        ddst.copy_(hsrc, non_blocking=True)
                g_in[gi].record(s_in)
                stream.wait_event(g_in[gi])
                if started[gi]:
                    stream.wait_event(g_out[gi])    # outputs are free once last step's copies ran
                for i in idxs:
                    calls[i][6]()
                g_cmp[gi].record(stream)
                s_out.wait_event(g_cmp[gi])
                with torch.cuda.stream(s_out):
                    for dsrc, hdst in d2h:
                        hdst.copy_(dsrc, non_blocking=True)
                g_out[gi].record(s_out)
                started[gi] = True

        for _ in range(max(1, min(args.warmup, 2))):
            e2e_step()
        torch.cuda.synchronize()
        e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        ke = max(1, min(args.steps, 10))
        barrier()
        torch.cuda.synchronize()
        e0.record(stream)
        s_in.wait_stream(stream)
        s_out.wait_stream(stream)
        for _ in range(ke):
            e2e_step()
        stream.wait_stream(s_in)
        stream.wait_stream(s_out)
        e1.record(stream)
        torch.cuda.synchronize()
        barrier()
        e2e_ms = e0.elapsed_time(e1) / ke
        h2d_bytes = sum(h.numel() * h.element_size() for g in groups for h, _ in g[0])
        d2h_bytes = sum(h.numel() * h.element_size() for g in groups for _, h in g[2])

    # the same step as one CUDA graph, replayed: no launch gaps, L2 warm
    # from call to call (the number small, launch-bound layers reach when a
    # framework replays them in a graph); not the headline
    graph_ms, graph_info = None, None
    if not args.no_graph:
        graph_ms, graph_info = graph_replay_ms(calls, stream, ms_per_step)

    ms_per_step, e2e_ms, graph_ms = max_over_ranks([ms_per_step, e2e_ms, graph_ms], dist, dev)

    hbm_peak, hbm_kind, tc_peak, tc_kind = peaks
    fams = {}
    passes = {}
    for i, c in enumerate(calls):
        ms = statistics.mean(per_call[k][i] for k in range(args.steps))
        for key, dct in ((f"{c[0]}:{c[2]}", fams), (c[0], passes)):
            f = dct.setdefault(key, {"ms": 0.0, "bytes": 0, "fma": 0, "launches": 0, "calls": 0})
            f["ms"] += ms
            f["bytes"] += c[3]
            f["fma"] += c[4]
            f["launches"] += c[5]
            f["calls"] += 1
    per_layer = {}
    for i, c in enumerate(calls):
        ms = statistics.median(per_call[k][i] for k in range(args.steps))
        per_layer.setdefault(c[1], {})[c[0]] = {"plan": c[2].split(":")[0], "us": round(ms * 1e3, 2),
                                                "GBps": round(c[3] / ms / 1e6, 1),
                                                "TFLOPs": round(2 * c[4] / ms / 1e9, 2)}
    fma_src = ("measured in this run (register-only FP32 FMA probe, dwconv_fma_probe; nominal "
               "152 SMs x 128 lanes x 2 FLOP x 2.07 GHz = 80.5 TFLOP/s)")
    tc_src = (f"{tc_kind} ({'MEASURED_PEAKS.json bf16_tflops (dense bf16 burst; fp16 has the same dense rate)' if tc_kind == 'measured' else 'profiling recipe fallback 1.9 PFLOP/s'})")
    rl = {}
    for key, f in fams.items():
        pass_, plan, dt = key.split(":")
        family = plan.replace("multi-", "")
        if family in ("ibgemm", "tcwgrad", "septc", "ibgemm-cached"):
            bp = ("tensor", tc_peak, tc_src)
        elif fma_tflops:
            bp = ("alu", fma_tflops, fma_src)
        else:
            bp = ("alu", 80.5, "nominal FP32 FMA rate (152 x 128 x 2 x 2.07 GHz)")
        te = ncu_traffic(f"{name}:{key}", family)
        r = roofline_of(f, bp, hbm_peak, hbm_kind, te)
        if te:
            r["traffic_layer"] = te.get("layer")
            r["traffic_layer_algorithmic_bytes"] = te.get("algorithmic_bytes_per_launch")
        r.update({"kernel": key, "calls": f["calls"], "launches": f["launches"], "ms": round(f["ms"], 4),
                  "share": round(f["ms"] / ms_per_step, 4)})
        rl[key] = r
    dom = max(fams, key=lambda k: fams[k]["ms"])
    unit = "TFLOP/s" if name in ("largek", "largek_infer") else "GB/s"

    def metric_of(ms):
        return job_throughput(world, step_fma if unit == "TFLOP/s" else step_bytes, ms, unit)

    dts = sorted({getattr(i, "dtype", "f32") for i in items}, key=lambda d: ("f32", "f16", "bf16").index(d))
    rec = {
        "workload": WORKLOAD_TEXT[name], "name": name,
        "value": round(metric_of(ms_per_step), 3), "unit": unit,
        "ms_per_step": round(ms_per_step, 4),
        "GBps": round(job_throughput(world, step_bytes, ms_per_step, "GB/s"), 1),
        "TFLOPs_valid": round(job_throughput(world, step_fma, ms_per_step, "TFLOP/s"), 3),
        "dtype": "+".join(dts),
        "step_bytes": step_bytes, "step_fma_valid": step_fma,
        "step_fma_dense": step_fma_dense, "valid_over_dense": round(step_fma / step_fma_dense, 4),
        "TFLOPs_dense": round(job_throughput(world, step_fma_dense, ms_per_step, "TFLOP/s"), 3),
        "roofline": rl[dom],
        "roofline_by_family": rl,
        "passes": {k: {"ms": round(v["ms"], 4), "GBps": round(v["bytes"] / v["ms"] / 1e6, 1),
                       "TFLOPs_valid": round(2 * v["fma"] / v["ms"] / 1e9, 3), "launches": v["launches"],
                       "share": round(v["ms"] / ms_per_step, 4)}
                   for k, v in passes.items()},
        "per_layer": per_layer,
        "gpu_launches": launches_per_step * args.steps,
        "e2e": ({"value": round(metric_of(e2e_ms), 3), "unit": unit, "ms_per_step": round(e2e_ms, 4),
                 "h2d_bytes_per_step": h2d_bytes, "d2h_bytes_per_step": d2h_bytes,
                 "copies": "per layer: H2D on one side stream, D2H on another, overlapped with other layers' compute"}
                if e2e_ms else None),
        "graph_replay": ({"value": round(metric_of(graph_ms), 3), "unit": unit, "ms_per_step": round(graph_ms, 4),
                          "replays": graph_info,
                          "l2": "warm: the step's calls back to back in one graph, no flush between them"}
                         if graph_ms else ({"error": graph_info} if graph_info else None)),
        "clocks": clock_summary(clk.lines),
        "clock_lines": clk.lines,
        "wall_s_timed": round(t_wall, 3),
        "steps": args.steps,
    }
    del calls, groups, hc, out_host, flush, flush_clean
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    return rec


def gpu_arm(args, names, rank, world):
    import torch
    from depthwise_convolution_dwconv2d_gb300 import binding as B, build as BLD

    BLD.build()
    B.load()
    dev = torch.device("cuda", int(os.environ.get("LOCAL_RANK", 0)))
    torch.cuda.set_device(dev)
    # a stream of its own (not the legacy default stream), current for every
    # torch op too, so that the step can also be captured as a CUDA graph
    stream = torch.cuda.Stream(device=dev)
    torch.cuda.set_stream(stream)
    dist = None
    if world > 1:
        import torch.distributed as dist_
        dist = dist_
    peaks = load_peaks()
    fma_tflops = fma_probe_tflops(dev, stream)
    recs, items_of = {}, {}
    for name in names:
        items = build_workload(name)
        if args.layers:
            keep = set(args.layers.split(","))
            items = [i for i in items if i.label() in keep]
            if not items:
                continue
        if args.batch:
            # smaller batch of the same layers (profiling runs only)
            items = [type(i)(**{**i.__dict__, "N": args.batch}) for i in items]
        items_of[name] = items
        recs[name] = time_workload(name, items, args, dev, stream, world, dist, peaks, fma_tflops)
    if not recs:
        raise SystemExit(f"--layers {args.layers} matched nothing")
    return recs, items_of, fma_tflops, peaks


def summary(r):
    """A workload's figures for the metric line. The whole record (every family's roofline, every layer) is some
    thousand characters a workload: with all of them the line had 43 KB and was read back cut. It goes to stderr."""
    pick = lambda d, *keys: {k: d[k] for k in keys if d and k in d}  # noqa: E731
    return {**pick(r, "value", "unit", "ms_per_step", "dtype", "gpu_launches"),
            "roofline": pick(r.get("roofline"), "bound", "achieved", "unit", "frac", "kernel", "share"),
            "e2e": (r.get("e2e") or {}).get("value"), "graph_replay_ms": (r.get("graph_replay") or {}).get("ms_per_step"),
            "cpu_value": (r.get("cpu_baseline") or {}).get("value")}


def metric_line(args, recs, head, world, fma_tflops):
    """The one line: the headline workload's figures, the others in short."""
    h = recs[head]
    head_clocks = clock_summary(h["clock_lines"])
    lines = [ln for r in recs.values() for ln in r["clock_lines"]]
    return {
        "metric": METRIC, "value": h["value"], "unit": h["unit"], "n_gpus": world, "steps": args.steps,
        "warmup": args.warmup, "ms_per_step": h["ms_per_step"], "higher_is_better": True,
        "scaling": "weak", "vs_baseline": None, "dtype": h["dtype"],
        "data": "synthetic (SplitMix64 + Box-Muller, seed 0)",
        "config": {"workload": h["workload"], "name": head,
                   **({"layers": args.layers} if args.layers else {}),
                   **({"batch_override": args.batch} if args.batch else {}),
                   "parallelism": f"replicas x{world} (no collective)",
                   "l2": "flushed before every call (2x L2 written, then a clean 2x L2 buffer read: inputs "
                         "not cached, no dirty lines left); inputs resident in HBM",
                   "step_bytes": h["step_bytes"], "step_fma_valid": h["step_fma_valid"],
                   "GBps": h["GBps"], "tflops_valid": h["TFLOPs_valid"]},
        "roofline": h["roofline"],
        "e2e": h["e2e"],
        "gpu_launches": h["gpu_launches"],
        "gpu_launches_all_workloads": sum(r["gpu_launches"] for r in recs.values()),
        "clocks": head_clocks or clock_summary(lines),
        "clocks_all_workloads": clock_summary(lines),
        "fp32_fma_probe_tflops": round(fma_tflops, 2),
        **({"cpu_baseline": h["cpu_baseline"]} if "cpu_baseline" in h else {}),
        "configs": {n: summary(r) for n, r in recs.items()},
    }


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--gpus", type=int, default=1)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--warmup", type=int, default=3)
    ap.add_argument("--impl", default="gb300", choices=["gb300", "reference"])
    ap.add_argument("--workload", default="all", choices=["all"] + list(ORDER))
    ap.add_argument("--no-e2e", action="store_true")
    ap.add_argument("--no-cpu-baseline", action="store_true")
    ap.add_argument("--no-graph", action="store_true", help="skip the CUDA-graph replay of each step")
    ap.add_argument("--cpu-seconds", type=float, default=8.0)
    ap.add_argument("--layers", default="", help="comma-separated layer labels to keep (profiling runs)")
    ap.add_argument("--batch", type=int, default=0, help="override the batch size (profiling runs)")
    args = ap.parse_args()
    names = list(ORDER) if args.workload == "all" else [args.workload]
    head = HEADLINE if HEADLINE in names else names[0]
    rank = int(os.environ.get("RANK", 0))
    world = int(os.environ.get("WORLD_SIZE", 1))
    unit_of = lambda n: "TFLOP/s" if n in ("largek", "largek_infer") else "GB/s"

    if args.impl == "reference":
        if rank != 0:
            return
        items = build_workload(head)
        total = max(1, args.steps + args.warmup)
        per_step = max(1.0, min(args.cpu_seconds, 150.0 / total))
        vals, desc, t_all = [], "", 0.0
        for k in range(total):
            cb = cpu_baseline(head, items, per_step, unit_of(head))
            desc = cb["sample"]
            if k >= args.warmup:
                vals.append(cb["value"])
        v = statistics.mean(vals)
        line = {"metric": METRIC, "value": round(v, 5), "unit": unit_of(head), "n_gpus": 1, "steps": args.steps,
                "warmup": args.warmup, "higher_is_better": True, "scaling": "weak", "vs_baseline": None,
                "dtype": "f64", "data": "synthetic (SplitMix64 + Box-Muller, seed 0)", "impl": "reference",
                "config": {"workload": WORKLOAD_TEXT[head], "name": head},
                "cpu_baseline": {"value": round(v, 5), "unit": unit_of(head), "cores": cb["cores"],
                                 "cpu_model": cb["cpu_model"], "kind": "oracle", "sample": desc},
                "e2e": {"value": round(v, 5), "unit": unit_of(head), "h2d_bytes_per_step": 0,
                        "d2h_bytes_per_step": 0}}
        print(json.dumps(line))
        return

    if world > 1:
        import torch
        import torch.distributed as dist
        torch.cuda.set_device(int(os.environ.get("LOCAL_RANK", 0)))
        dist.init_process_group("nccl")
    recs, items_of, fma_tflops, peaks = gpu_arm(args, names, rank, world)
    if rank == 0:
        head = head if head in recs else next(iter(recs))
        if not args.no_cpu_baseline:
            for n in recs:
                recs[n]["cpu_baseline"] = cpu_baseline(n, items_of[n], args.cpu_seconds, recs[n]["unit"])
        print("details: " + json.dumps({n: {k: v for k, v in r.items() if k != "clock_lines"} for n, r in recs.items()}),
              file=sys.stderr, flush=True)
        print(json.dumps(metric_line(args, recs, head, world, fma_tflops)))
    if world > 1:
        import torch.distributed as dist
        dist.destroy_process_group()


if __name__ == "__main__":
    main()
