"""Throughput of the fused, chunked top-K KL loss (forward + backward) on one MI355X.

One step = one kd_chunked_kl_fwd_bwd call over the whole batch (every chunk: forward
GEMM + logsumexp + exp(z - max), gather, loss, dz from the kept exponentials, sparse
correction, dh and dW GEMMs) with inputs already resident in HBM.  Prints one JSON line.

Default workload: N=32768 tokens, d=3072, V=128256, K=100, chunk 2048, bf16, packed
sequences with each sequence's first token masked (synthetic, seeded).
"""
import argparse
import dataclasses
import hashlib
import json
import os
import sys
import time

import numpy as np

ROOT = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, ROOT)

PEAK_BF16_TFLOPS = 2500.0   # MI355X dense bf16 MFMA
PEAK_F32_TFLOPS = 157.3     # MI355X dense fp32 MFMA
PEAK_HBM_GBS = 8000.0
GEMM_CLASSES = ("fwd_gemm_lse", "bwd_gemm_dz", "dh_gemm", "dw_gemm")


class ClockSampler:
    """While active, samples the GPU's current graphics clock and socket power through
    amd-smi every `period` seconds in a thread; `result()` gives their medians and range
    over the samples, or None where amd-smi is not available (one GPU visible to it only).
    The reading lags and some boxes report an idle value under load, so the bench line's
    clock_observed comes from in-kernel counters (unit_clocks) and this is kept beside it."""

    def __init__(self, period=0.005):
        self.period, self.mhz, self.watts, self._stop = period, [], [], None

    def __enter__(self):
        import threading
        try:
            import amdsmi
            amdsmi.amdsmi_init()
            hs = amdsmi.amdsmi_get_processor_handles()
            if len(hs) != 1:
                amdsmi.amdsmi_shut_down()
                return self
        except Exception:  # amd-smi missing or not permitted: no clock figure
            return self
        self._smi, self._h = amdsmi, hs[0]
        self._stop = threading.Event()

        def loop():
            while not self._stop.is_set():
                try:
                    self.mhz.append(float(self._smi.amdsmi_get_clock_info(
                        self._h, self._smi.AmdSmiClkType.GFX)["clk"]))
                    self.watts.append(float(self._smi.amdsmi_get_power_info(
                        self._h)["current_socket_power"]))
                except Exception:
                    pass
                self._stop.wait(self.period)

        self._thread = threading.Thread(target=loop, daemon=True)
        self._thread.start()
        return self

    def __exit__(self, *exc):
        if self._stop is not None:
            self._stop.set()
            self._thread.join()
            try:
                self._smi.amdsmi_shut_down()
            except Exception:
                pass
        return False

    def result(self):
        if not self.mhz:
            return None
        return {"gfx_mhz_median": round(float(np.median(self.mhz)), 1),
                "gfx_mhz_min": round(float(np.min(self.mhz)), 1),
                "gfx_mhz_max": round(float(np.max(self.mhz)), 1),
                "socket_power_w_median": (round(float(np.median(self.watts)), 1)
                                          if self.watts else None),
                "samples": len(self.mhz),
                "source": "amd-smi current graphics clock and socket power, sampled every 5 ms "
                          "over the timed steps (the reading changes slowly; indicative only)"}


CLOCK_GROUPS = 2048   # one-wave workgroups per clock stamp: eight per compute unit


def unit_clocks(before, after, khz):
    """Average shader clock in MHz of each compute unit between two kd_clock_stamp records
    (int64 arrays of 3 * n_groups words).  Stamps are paired unit by unit: the cycle
    counters of different units are not aligned with each other."""
    def per_unit(rec):
        out = {}
        for ident, cyc, tick in np.asarray(rec, dtype=np.int64).reshape(-1, 3).tolist():
            out.setdefault(((ident >> 32) & 15, (ident >> 8) & 0xFF), (cyc, tick))
        return out
    a, b = per_unit(before), per_unit(after)
    return np.array([(b[k][0] - c0) / (b[k][1] - t0) * khz / 1000.0
                     for k, (c0, t0) in a.items() if k in b and b[k][1] > t0])


def warm_up(step, n, seconds=0.5):
    """At least n untimed calls of step, and calls for at least `seconds` of wall time:
    a few short steps do not bring the GPU to its steady clock."""
    import torch
    t0 = time.perf_counter()
    k = 0
    while k < n or time.perf_counter() - t0 < seconds:
        out = step()
        del out
        k += 1
        if k % 8 == 0:
            torch.cuda.synchronize()
    torch.cuda.synchronize()
    return k


def timed_steps(step, steps):
    """`steps` calls of step, each bracketed by device synchronisations: (list of ms per
    call, the last call's output).  The previous call's outputs go back to the pool before
    the next call, so peak memory is that of one call."""
    import torch
    out = None
    times = []
    torch.cuda.synchronize()
    for _ in range(steps):
        out = None
        t0 = time.perf_counter()
        out = step()
        torch.cuda.synchronize()
        times.append((time.perf_counter() - t0) * 1e3)
    return times, out


def timed_then_profiled(step, steps):
    """Time `steps` calls of step with nothing else recorded (median of the calls), then
    run them again with the library's per-launch HIP events on: (ms per call, kernel table
    of that pass)."""
    import torch

    import output_head_kl_amd as kd
    times, _ = timed_steps(step, steps)
    ms = float(np.median(times))
    # recorded steps first, discarded, for at least 0.5 s: they fill the library's pool
    # of HIP events and bring the GPU back to its steady clock under the recording
    kd.profile_read()
    kd.profile_enable(True)
    warm_up(step, 1)
    kd.profile_read()
    for _ in range(steps):
        step()
    torch.cuda.synchronize()
    kd.profile_enable(False)
    return ms, _kernel_table(kd.profile_read(), steps)


def parse():
    ap = argparse.ArgumentParser()
    ap.add_argument("--gpus", type=int, default=1)
    ap.add_argument("--steps", type=int, default=5)
    ap.add_argument("--warmup", type=int, default=2)
    ap.add_argument("--config", type=int, default=2, help="workload id (synth.CONFIGS)")
    ap.add_argument("--N", type=int, default=None, help="override the token count")
    ap.add_argument("--chunk", type=int, default=None, help="override the chunk size")
    ap.add_argument("--no-cpu-baseline", action="store_true")
    ap.add_argument("--cpu-rows", type=int, default=4096,
                    help="token rows of the workload timed through the CPU oracle (a bounded "
                         "sample: ~15-25 s of host time at the full vocabulary)")
    ap.add_argument("--no-reference", action="store_true",
                    help="skip the torch kernels timed for scale (gemm_reference of the fused "
                         "call, read_reference of --topk), e.g. so that a kernel trace holds the "
                         "library's kernels only")
    ap.add_argument("--no-profile", action="store_true",
                    help="skip per-kernel HIP-event timing inside the timed region")
    ap.add_argument("--split", action="store_true",
                    help="time the forward half (kd_chunked_kl_fwd) and the backward half "
                         "(kd_chunked_kl_bwd) separately instead of the fused call; prints one "
                         "JSON line")
    ap.add_argument("--shard", type=int, default=0,
                    help="time one GPU's share of a vocabulary-sharded head: rows [0, V/G) of W "
                         "with the full token batch (forward statistics + backward); G = value")
    ap.add_argument("--torch-baselines", action="store_true",
                    help="context only: peak memory, time and loss of a dense and a "
                         "forward-chunked PyTorch implementation of the same loss (torch "
                         "autograd, hipBLASLt GEMMs) next to the fused library call, "
                         "N = 4K..256K; prints one JSON line")
    ap.add_argument("--topk", action="store_true",
                    help="time the teacher top-K cache producer (kd_teacher_topk) on N=32768 rows "
                         "of V=128256 bf16 teacher logits, K=100; prints one JSON line")
    ap.add_argument("--memory-sweep", action="store_true",
                    help="measure peak device memory of one call and the steady time per call "
                         "for N = 4K .. 256K tokens (d=3072, V=128256, K=100, chunk 4096) and "
                         "fit peak = a + b*N; prints one JSON line and exits")
    ap.add_argument("--dw-group-tokens", type=int, default=None,
                    help="allocate the workspace for dW groups of at most this many tokens "
                         "(0 = one chunk, the smallest workspace); default 16384")
    ap.add_argument("--no-small-workspace", action="store_true",
                    help="skip the second measurement with the smallest workspace (dW "
                         "accumulated one chunk at a time: no buffer beyond one chunk of logits)")
    ap.add_argument("--autograd", action="store_true",
                    help="time the loss as a torch autograd function (chunked_kl_loss forward + "
                         "backward), in its fused mode and in its recompute mode; prints one "
                         "JSON line")
    ap.add_argument("--copy-gib", type=float, default=0.0,
                    help="after the run, launch one plain device copy of this many GiB "
                         "(a kernel of known traffic, for scaling HBM byte counters)")
    return ap.parse_args()


def kernel_source_hash(files=("kd_gemm.h", "kd_kernels.hip", "kd_api.hip",
                              "kd_internal.h")):
    """Hash of the sources that the counters were taken on, comments and whitespace
    removed: a change of the code (not of its comments) makes the record stale."""
    import re
    h = hashlib.sha256()
    for f in files:
        with open(os.path.join(ROOT, "output_head_kl_amd", "csrc", f), encoding="utf-8") as fh:
            src = fh.read()
        src = re.sub(r"/\*.*?\*/", " ", src, flags=re.S)     # block comments
        src = re.sub(r"//[^\n]*", " ", src)                   # line comments
        h.update(" ".join(src.split()).encode())
    return h.hexdigest()[:16]


def traffic_for(kernel, workload):
    """Counter-derived HBM bytes per launch recorded under profiles/, if the kernels have
    not changed since the counters were taken."""
    path = os.path.join(ROOT, "profiles", "traffic.json")
    if not os.path.exists(path):
        return None
    rec = json.load(open(path))
    if rec.get("source_hash") != kernel_source_hash() or rec.get("workload") != workload:
        return None
    k = rec.get("kernels", {}).get(kernel)
    return None if k is None else k.get("hbm_bytes_per_launch")


def cpu_baseline(inp, rows):
    import oracle
    import synth
    try:
        from threadpoolctl import threadpool_info
        threads = max([t.get("num_threads", 1) for t in threadpool_info()] or [1])
    except Exception:  # pragma: no cover
        threads = os.cpu_count()
    sel = synth.subset_rows(inp.cfg, inp.seed, rows)
    sub = synth.take_rows(inp, sel)
    h64, W64 = sub.h64(), sub.W64()
    t0 = time.perf_counter()
    oracle.forward_backward(h64, W64, sub.idx, sub.p, sub.mask, block_rows=128)
    dt = time.perf_counter() - t0
    return {"value": len(sel) / dt, "unit": "tokens/s", "cores": int(threads), "kind": "oracle",
            "sample": f"{len(sel)} seeded token rows of the same workload (full V and d), "
                      f"float64 numpy, loss + dh + dW, {dt:.1f} s"}


def topk_traffic(workload):
    """HBM bytes per launch of the top-K kernel recorded under profiles/, if current."""
    path = os.path.join(ROOT, "profiles", "traffic_topk.json")
    if not os.path.exists(path):
        return None
    rec = json.load(open(path))
    if (rec.get("source_hash") != kernel_source_hash(("kd_topk.hip", "kd_internal.h"))
            or rec.get("workload") != workload):
        return None
    return rec.get("hbm_bytes_per_launch")


def read_reference(torch, x, N, V, kern_ms):
    """torch's row sum over the teacher logits (a plain streaming read of the same bytes):
    median of 10 HIP-event-timed calls after 0.5 s of calls."""
    ref = lambda: x.sum(dim=1, dtype=torch.float32)
    warm_up(ref, 20)
    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    rs = []
    for _ in range(10):
        e0.record()
        ref()
        e1.record()
        torch.cuda.synchronize()
        rs.append(e0.elapsed_time(e1))
    ref_ms = float(np.median(rs))
    ref_gbs = N * V * 2 / (ref_ms * 1e-3) / 1e9
    return {"op": "torch sum(logits, dim=1, dtype=float32), same tensor",
            "ms": round(ref_ms, 4), "GB/s": round(ref_gbs, 1),
            "producer_rate_over_it": round(ref_ms / kern_ms, 4)}


def bench_topk(args):
    """Teacher top-K cache producer: one row of logits per token, read once (HBM-bound)."""
    import torch

    import output_head_kl_amd as kd
    import synth
    N, V, K = args.N or 32768, 128256, 100
    seed = synth.BASE_SEED + 10
    t0 = time.perf_counter()
    bits = synth.make_teacher_logits(N, V, seed=seed, threads=16)
    print(f"[bench] generated teacher logits N={N} V={V} in {time.perf_counter() - t0:.1f} s",
          file=sys.stderr, flush=True)
    x = torch.from_numpy(bits.view(np.int16)).cuda().view(torch.bfloat16)
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    idx = torch.empty((N, K), dtype=torch.int32, device="cuda")
    pr = torch.empty((N, K), dtype=torch.float32, device="cuda")
    lse = torch.empty(N, dtype=torch.float32, device="cuda")
    lib = kd._lib()
    strm = torch.cuda.current_stream().cuda_stream

    def call():
        kd._check(lib.kd_teacher_topk(x.data_ptr(), kd.KD_BF16, N, V, K, idx.data_ptr(),
                                      pr.data_ptr(), lse.data_ptr(), ws.data_ptr(), 256, strm))

    warm_up(call, args.warmup)
    ms, kt = timed_then_profiled(call, args.steps)
    kern_ms = kt["teacher_topk"]["avg_ms"]
    algo_bytes = N * V * 2 + N * K * 8 + N * 4       # logits once; idx, p and lse written
    achieved = algo_bytes / (kern_ms * 1e-3) / 1e9
    workload = f"teacher_topk_N{N}_V{V}_K{K}_bf16"
    res = {
        "metric": "tokens/s, teacher top-K cache producer (top-100 probabilities per position)",
        "value": round(N / (ms * 1e-3), 1), "unit": "tokens/s", "n_gpus": 1, "steps": args.steps,
        "warmup": args.warmup, "ms_per_step": round(ms, 3), "higher_is_better": True,
        "scaling": "weak", "vs_baseline": None, "dtype": "bf16", "data": "synthetic",
        "config": {"workload": workload, "N": N, "V": V, "K": K},
        "roofline": {"bound": "hbm", "kernel": "teacher_topk", "achieved": round(achieved, 1),
                     "peak": PEAK_HBM_GBS, "unit": "GB/s", "frac": round(achieved / PEAK_HBM_GBS, 4),
                     "traffic": topk_traffic(workload)},
        "kernels": kt, "cpu_baseline": None,
    }
    # For scale: a plain streaming read of the same logits by torch (a row sum), timed the
    # same way, after the measured calls.
    if not args.no_reference:
        try:  # context only: a failure here leaves the line whole
            res["read_reference"] = read_reference(torch, x, N, V, kern_ms)
        except Exception as e:  # noqa: BLE001
            res["read_reference"] = {"error": f"{type(e).__name__}: {e}"}
    if args.copy_gib > 0:
        n = int(args.copy_gib * 2**30) // 4
        src = torch.ones(n, dtype=torch.float32, device="cuda")
        dst = torch.empty_like(src)
        torch.cuda.synchronize()
        dst.copy_(src)
        torch.cuda.synchronize()
        del src, dst
    if not args.no_cpu_baseline:
        from oracle.topk import topk_probs
        try:
            from threadpoolctl import threadpool_info
            threads = max([t.get("num_threads", 1) for t in threadpool_info()] or [1])
        except Exception:  # pragma: no cover
            threads = os.cpu_count()
        rows = args.cpu_rows
        sub = synth.bf16_bits_to_f32(bits[:rows]).astype(np.float64)
        t0 = time.perf_counter()
        topk_probs(sub, K)
        dt = time.perf_counter() - t0
        res["cpu_baseline"] = {"value": rows / dt, "unit": "tokens/s", "cores": int(threads),
                               "kind": "oracle",
                               "sample": f"the first {rows} rows of the same logits, float64 numpy "
                                         f"(full-row stable sort), {dt:.1f} s"}
    print(json.dumps(res), flush=True)


def torch_baselines():
    """The loss written with torch ops, as a dense and as a forward-chunked autograd graph,
    for the pages' memory comparison (output head only), beside the fused library call, for
    N = 4K .. 256K tokens.  Per N and implementation: peak device memory of one call
    (forward and backward), the steady time per call, and the loss, which must equal the
    library's (each graph computes the same mean loss on the same inputs; the torch graphs
    round the logits to bf16 in their matrix product, the library keeps them in fp32).  Not
    part of the library: these run torch's kernels."""
    import torch

    import output_head_kl_amd as kd
    d, V, K, chunk = 3072, 128256, 100, 2048
    g = torch.Generator(device="cuda").manual_seed(20260804)
    W0 = torch.randn(V, d, device="cuda", generator=g, dtype=torch.bfloat16) * (2.0 / d ** 0.5)

    def loss_of(hc, W, idx, p, mask, count):
        z = torch.mm(hc, W.t()).float()
        lq = torch.log_softmax(z, dim=-1).gather(1, idx.long())
        ell = (torch.xlogy(p, p) - p * lq).sum(1)
        return (ell * mask).sum() / count

    results = []
    for N in [4096, 16384, 32768, 65536, 131072, 262144]:
        h0 = torch.randn(N, d, device="cuda", generator=g, dtype=torch.bfloat16)
        idx = torch.randint(0, V, (N, K), device="cuda", generator=g, dtype=torch.int32)
        p = torch.rand(N, K, device="cuda", generator=g) / K
        mask = torch.ones(N, device="cuda")
        row = {"N": N}
        for kind in ["fused_library", "forward_chunked", "dense"]:
            def call():
                if kind == "fused_library":
                    out = kd.fwd_bwd(h0, W0, idx, p, mask.to(torch.uint8), chunk=chunk)
                    return float(out[0].item())
                h = h0.detach().requires_grad_(True)
                W = W0.detach().requires_grad_(True)
                if kind == "dense":
                    loss = loss_of(h, W, idx, p, mask, float(N))
                else:  # chunks in the forward; autograd keeps every chunk's logits
                    loss = sum(loss_of(h[c:c + chunk], W, idx[c:c + chunk], p[c:c + chunk],
                                       mask[c:c + chunk], float(N))
                               for c in range(0, N, chunk))
                loss.backward()
                val = float(loss.detach().item())
                del loss, h, W
                return val
            torch.cuda.synchronize()
            torch.cuda.empty_cache()
            torch.cuda.reset_peak_memory_stats()
            try:
                t0 = time.perf_counter()
                loss_val = call()          # first call: peak memory (and warm-up)
                torch.cuda.synchronize()
                first_s = time.perf_counter() - t0
                peak = torch.cuda.max_memory_allocated()
                reps = 3 if first_s < 2.0 else 1
                times = []
                for _ in range(reps):     # steady time per call
                    t0 = time.perf_counter()
                    call()
                    torch.cuda.synchronize()
                    times.append(time.perf_counter() - t0)
                row[kind] = {"peak_gib": round(peak / 2**30, 3),
                             "s_per_call": round(float(np.median(times)), 4),
                             "tokens_per_s": round(N / float(np.median(times)), 1),
                             "loss": loss_val}
            except torch.cuda.OutOfMemoryError:
                row[kind] = "out of memory"
            torch.cuda.empty_cache()
            print(f"[baselines] N={N} {kind}: {row[kind]}", file=sys.stderr, flush=True)
        ref = row["fused_library"]["loss"] if isinstance(row.get("fused_library"), dict) else None
        for kind in ["forward_chunked", "dense"]:
            if isinstance(row.get(kind), dict) and ref is not None:
                row[kind]["loss_rel_diff_vs_library"] = abs(row[kind]["loss"] - ref) / abs(ref)
        results.append(row)
        del h0, idx, p, mask
    bad = [(r["N"], k, r[k]["loss_rel_diff_vs_library"]) for r in results
           for k in ("forward_chunked", "dense")
           if isinstance(r.get(k), dict) and r[k]["loss_rel_diff_vs_library"] > 2e-3]
    print(json.dumps({"torch_baselines": {"d": d, "V": V, "K": K, "chunk": chunk, "dtype": "bf16",
                                          "loss_check": "every torch loss within 2e-3 of the "
                                                        "library's" if not bad else f"FAILED {bad}",
                                          "rows": results}}), flush=True)
    if bad:
        sys.exit(1)


def memory_sweep(dw_group_tokens=None):
    """Peak device memory of one fused call (inputs, outputs, workspace) against N.

    Inputs are generated directly in their storage types, so the peak holds only h, W,
    idx, p, mask, the outputs and the workspace.  The device's free-memory drop across
    the call is compared with the growth of torch's reserved pool: equal values show
    the library allocated nothing of its own.  ``dw_group_tokens`` sizes the workspace
    (None: the default 16384-token dW group; 0: one chunk)."""
    import torch

    import output_head_kl_amd as kd
    d, V, K, chunk = 3072, 128256, 100, 4096
    g = torch.Generator(device="cuda").manual_seed(20260804)
    Ns = [4096, 8192, 16384, 32768, 65536, 131072, 262144]
    W = torch.randn(V, d, device="cuda", generator=g, dtype=torch.bfloat16) * (2.0 / d ** 0.5)
    torch.cuda.synchronize()
    base = torch.cuda.memory_allocated()
    peaks, rows = [], []
    for N in Ns:
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        torch.cuda.reset_peak_memory_stats()
        h = torch.randn(N, d, device="cuda", generator=g, dtype=torch.bfloat16)
        idx = torch.randint(0, V, (N, K), device="cuda", generator=g, dtype=torch.int32)
        p = torch.rand(N, K, device="cuda", generator=g)
        p.mul_(1.0 / K)
        mask = torch.ones(N, dtype=torch.uint8, device="cuda")
        ws_bytes = kd.workspace_bytes(N, d, V, K, chunk, dw_group_tokens=dw_group_tokens)
        torch.cuda.synchronize()
        free0, _ = torch.cuda.mem_get_info()
        res0 = torch.cuda.memory_reserved()
        out = kd.fwd_bwd(h, W, idx, p, mask, chunk=chunk, dw_group_tokens=dw_group_tokens)
        torch.cuda.synchronize()
        free1, _ = torch.cuda.mem_get_info()
        res1 = torch.cuda.memory_reserved()
        peaks.append(torch.cuda.max_memory_allocated())
        largest = max(ws_bytes, N * d * 2, V * d * 4)   # workspace, dh, dW
        # iteration rate: steady time per call (the call above warmed up), workspace reused
        del out
        ws = torch.empty(ws_bytes, dtype=torch.uint8, device="cuda")
        step = lambda: kd.fwd_bwd(h, W, idx, p, mask, chunk=chunk, workspace=ws)
        warm_up(step, 1, seconds=0.3)
        times, out = timed_steps(step, 3)
        ms = float(np.median(times))
        rows.append({"N": N, "peak_bytes": peaks[-1], "workspace_bytes": ws_bytes,
                     "device_free_drop_bytes": free0 - free1,
                     "torch_reserved_growth_bytes": res1 - res0,
                     "largest_allocation_bytes": largest,
                     "dense_bf16_logits_bytes": N * V * 2,
                     "ms_per_call": round(ms, 3), "tokens_per_s": round(N / (ms * 1e-3), 1)})
        del h, idx, p, mask, out, ws
        print(f"[memory] N={N}: peak {peaks[-1] / 2**30:.3f} GiB, free drop "
              f"{(free0 - free1) / 2**20:.1f} MiB, reserved growth {(res1 - res0) / 2**20:.1f} MiB, "
              f"{ms:.2f} ms per call", file=sys.stderr, flush=True)
    def linfit(x, y):
        b, a = np.polyfit(x, y, 1)
        fit = a + b * x
        r2 = 1.0 - np.sum((y - fit) ** 2) / np.sum((y - y.mean()) ** 2)
        return a, b, r2, float(np.abs(y - fit).max())

    # The workspace grows with N only until the dW group (16384 tokens) is full, then
    # stays constant: fit peak(N) over the points past that, and peak minus workspace
    # over all of them.
    x = np.array(Ns, dtype=np.float64)
    y = np.array(peaks, dtype=np.float64)
    ws = np.array([r["workspace_bytes"] for r in rows], dtype=np.float64)
    full = ws == ws.max()
    a, b, r2, resid = linfit(x[full], y[full])
    a2, b2, r22, resid2 = linfit(x, y - ws)
    res = {"memory_sweep": {"d": d, "V": V, "K": K, "chunk": chunk, "dtype": "bf16",
                            "dw_group_tokens": 16384 if dw_group_tokens is None else dw_group_tokens,
                            "W_bytes": V * d * 2, "allocated_before_sweep_bytes": base,
                            "fit_from_N": int(x[full].min()),
                            "fit_intercept_bytes": a, "fit_bytes_per_token": b, "r2": r2,
                            "max_abs_residual_bytes": resid,
                            "fit_without_workspace": {"intercept_bytes": a2,
                                                      "bytes_per_token": b2, "r2": r22,
                                                      "max_abs_residual_bytes": resid2},
                            "points": rows}}
    print(json.dumps(res), flush=True)


def gemm_reference(torch, h, W, cfg, fwd_ms):
    """For scale: torch's plain GEMM (hipBLASLt) on the forward GEMM's shape, one chunk of
    tokens against the whole W, bf16 in and out, with no epilogue at all (no logsumexp, no
    gather, no exponentials kept).  Both operand orders; median of 10 event-timed calls
    each, after 0.5 s of calls."""
    import torch.nn.functional as F
    hc = h[:cfg.chunk]
    forms = {"linear(W, h_c): [V, chunk] out": lambda: F.linear(W, hc),
             "linear(h_c, W): [chunk, V] out": lambda: F.linear(hc, W)}
    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    got = {}
    for name, fn in forms.items():
        warm_up(fn, 3)
        ts = []
        for _ in range(10):
            e0.record()
            fn()
            e1.record()
            torch.cuda.synchronize()
            ts.append(e0.elapsed_time(e1))
        got[name] = round(float(np.median(ts)), 4)
    best = min(got.values())
    flops = 2.0 * cfg.chunk * cfg.V * cfg.d
    return {"op": "torch.nn.functional.linear (hipBLASLt), bf16, one chunk, no epilogue",
            "ms": got, "best_tflops": round(flops / (best * 1e-3) / 1e12, 1),
            "fwd_gemm_lse_ms": round(fwd_ms, 4),
            "fwd_gemm_lse_speed_over_it": round(best / fwd_ms, 4)}


def _kernel_table(ktimes, steps):
    out = {}
    for name, (tot, n) in ktimes.items():
        if n:
            out[name] = {"total_ms_per_step": tot / steps, "launches_per_step": n / steps,
                         "avg_ms": tot / n}
    return out


def bench_split(args, kd, torch, cfg, h, W, idx, p, mask, ws):
    """Forward half and backward half timed separately (each over args.steps calls)."""
    g = torch.ones(1, dtype=torch.float32, device="cuda")
    loss, row_lse = kd.fwd(h, W, idx, p, mask, chunk=cfg.chunk, workspace=ws)
    def fwd_bwd_pair():
        kd.fwd(h, W, idx, p, mask, chunk=cfg.chunk, workspace=ws)
        kd.bwd(h, W, idx, p, row_lse, g, mask, chunk=cfg.chunk, workspace=ws)

    warm_up(fwd_bwd_pair, args.warmup)
    print("[bench] warmup done", file=sys.stderr, flush=True)
    res_half = {
        "fwd": timed_then_profiled(
            lambda: kd.fwd(h, W, idx, p, mask, chunk=cfg.chunk, workspace=ws), args.steps),
        "bwd": timed_then_profiled(
            lambda: kd.bwd(h, W, idx, p, row_lse, g, mask, chunk=cfg.chunk, workspace=ws),
            args.steps)}
    fwd_ms, fk = res_half["fwd"]
    bwd_ms, bk = res_half["bwd"]
    ms = fwd_ms + bwd_ms
    peak = PEAK_BF16_TFLOPS if cfg.dtype == "bf16" else PEAK_F32_TFLOPS
    gem = {k: v for k, v in bk.items() if k in GEMM_CLASSES}
    dom = max(gem, key=lambda k: gem[k]["total_ms_per_step"])
    achieved = 2.0 * cfg.N * cfg.V * cfg.d / gem[dom]["launches_per_step"] / (gem[dom]["avg_ms"] * 1e-3) / 1e12
    workload = f"fused_kl_split_fwd_bwd_N{cfg.N}_d{cfg.d}_V{cfg.V}_K{cfg.K}_chunk{cfg.chunk}_{cfg.dtype}"
    res = {
        "metric": "tokens/s, fused KL as separate forward (kd_chunked_kl_fwd) and backward "
                  "(kd_chunked_kl_bwd) calls, N=32K d=3072 V=128256 K=100",
        "value": round(cfg.N / (ms * 1e-3), 1), "unit": "tokens/s", "n_gpus": 1,
        "steps": args.steps, "warmup": args.warmup, "ms_per_step": round(ms, 3),
        "higher_is_better": True, "scaling": "weak", "vs_baseline": None, "dtype": cfg.dtype,
        "data": "synthetic",
        "config": {"workload": workload, "N": cfg.N, "d": cfg.d, "V": cfg.V, "K": cfg.K,
                   "chunk": cfg.chunk, "mask": cfg.mask},
        "fwd_ms": round(fwd_ms, 3), "bwd_ms": round(bwd_ms, 3),
        "fwd_tflops_2NVd": round(2.0 * cfg.N * cfg.V * cfg.d / (fwd_ms * 1e-3) / 1e12, 1),
        "bwd_tflops_6NVd": round(6.0 * cfg.N * cfg.V * cfg.d / (bwd_ms * 1e-3) / 1e12, 1),
        "roofline": {"bound": "mfma", "kernel": dom, "achieved": round(achieved, 1), "peak": peak,
                     "unit": "TFLOP/s", "frac": round(achieved / peak, 4), "traffic": None},
        "kernels_fwd": fk, "kernels_bwd": bk, "cpu_baseline": None,
    }
    print(json.dumps(res), flush=True)


def bench_autograd(args, kd, torch, cfg, h, W, idx, p, mask):
    """The loss as a torch autograd function of h and W: forward and backward of
    chunked_kl_loss, in its fused mode (one-call loss and gradients held for the backward)
    and in its recompute mode (the backward recomputes the logits)."""
    hg = h.detach().clone().requires_grad_(True)
    Wg = W.detach().clone().requires_grad_(True)
    res_modes = {}
    for mode in ("fused", "recompute"):
        def step():
            hg.grad = None
            Wg.grad = None
            loss = kd.chunked_kl_loss(hg, Wg, idx, p, mask, chunk=cfg.chunk, mode=mode)
            loss.backward()
            return loss.detach()

        warm_up(step, args.warmup)
        torch.cuda.synchronize()
        torch.cuda.reset_peak_memory_stats()
        times, loss = timed_steps(step, args.steps)
        ms = float(np.median(times))
        res_modes[mode] = {"ms_per_step": round(ms, 3), "tokens_per_s": round(cfg.N / (ms * 1e-3), 1),
                           "peak_mem_gib": round(torch.cuda.max_memory_allocated() / 2**30, 3),
                           "loss": float(loss)}
        print(f"[bench] autograd {mode}: {ms:.2f} ms per step", file=sys.stderr, flush=True)
    ms = res_modes["fused"]["ms_per_step"]
    peak = PEAK_BF16_TFLOPS if cfg.dtype == "bf16" else PEAK_F32_TFLOPS
    workload = f"fused_kl_autograd_N{cfg.N}_d{cfg.d}_V{cfg.V}_K{cfg.K}_chunk{cfg.chunk}_{cfg.dtype}"
    res = {
        "metric": "tokens/s, fused KL as a torch autograd function (chunked_kl_loss forward + "
                  "backward, fused mode), N=32K d=3072 V=128256 K=100",
        "value": res_modes["fused"]["tokens_per_s"], "unit": "tokens/s", "n_gpus": 1,
        "steps": args.steps, "warmup": args.warmup, "ms_per_step": ms,
        "higher_is_better": True, "scaling": "weak", "vs_baseline": None, "dtype": cfg.dtype,
        "data": "synthetic",
        "config": {"workload": workload, "N": cfg.N, "d": cfg.d, "V": cfg.V, "K": cfg.K,
                   "chunk": cfg.chunk, "mask": cfg.mask},
        "tflops_executed_6NVd": round(6.0 * cfg.N * cfg.V * cfg.d / (ms * 1e-3) / 1e12, 1),
        "frac_of_peak_executed": round(6.0 * cfg.N * cfg.V * cfg.d / (ms * 1e-3) / 1e12 / peak, 4),
        "modes": res_modes, "roofline": None, "cpu_baseline": None,
    }
    print(json.dumps(res), flush=True)


def bench_shard(args, kd, torch, cfg, h, W, idx, p, mask):
    """One vocabulary shard (rows [0, V/G) of W) over the whole token batch: the forward
    statistics and the backward, as one GPU of a G-way tensor-parallel head would run
    between its collectives (which are not part of this)."""
    G = args.shard
    Vs = (cfg.V + G - 1) // G
    Ws = W[:Vs].contiguous()
    # A shard has V/G vocabulary rows, so G times the workload's chunk keeps the chunk's
    # logits buffer (chunk x V_shard bf16) the size the unsharded call has; --chunk
    # overrides it.
    if args.chunk is None:
        cfg = dataclasses.replace(cfg, chunk=min(cfg.chunk * G, cfg.N))
    ws = torch.empty(kd.workspace_bytes(cfg.N, cfg.d, Vs, cfg.K, cfg.chunk,
                                        kd.KD_BF16 if cfg.dtype == "bf16" else kd.KD_F32),
                     dtype=torch.uint8, device="cuda")
    lse = torch.full((cfg.N,), 14.0, dtype=torch.float32, device="cuda")   # stands in for the
    g = torch.ones(1, dtype=torch.float32, device="cuda")                  # combined logsumexp

    def step():
        kd.vocab_shard_fwd(h, Ws, idx, p, 0, cfg.V, chunk=cfg.chunk, workspace=ws)
        kd.vocab_shard_bwd(h, Ws, idx, p, lse, 0, cfg.V, g, mask, chunk=cfg.chunk, workspace=ws)

    warm_up(step, args.warmup)
    ms, kt = timed_then_profiled(step, args.steps)
    peak = PEAK_BF16_TFLOPS if cfg.dtype == "bf16" else PEAK_F32_TFLOPS
    gem = {k: v for k, v in kt.items() if k in GEMM_CLASSES}
    dom = max(gem, key=lambda k: gem[k]["total_ms_per_step"])
    achieved = 2.0 * cfg.N * Vs * cfg.d / gem[dom]["launches_per_step"] / (gem[dom]["avg_ms"] * 1e-3) / 1e12
    res = {
        "metric": f"tokens/s of one GPU's share of a {G}-way vocabulary-sharded head "
                  f"(forward statistics + backward, collectives excluded)",
        "value": round(cfg.N / (ms * 1e-3), 1), "unit": "tokens/s", "n_gpus": 1,
        "steps": args.steps, "warmup": args.warmup, "ms_per_step": round(ms, 3),
        "higher_is_better": True, "scaling": "weak", "vs_baseline": None, "dtype": cfg.dtype,
        "data": "synthetic",
        "config": {"workload": f"vocab_shard_{G}_N{cfg.N}_d{cfg.d}_Vshard{Vs}_K{cfg.K}_chunk{cfg.chunk}_{cfg.dtype}",
                   "N": cfg.N, "d": cfg.d, "V": cfg.V, "V_shard": Vs, "K": cfg.K, "chunk": cfg.chunk},
        "tflops_8NVsd": round(8.0 * cfg.N * Vs * cfg.d / (ms * 1e-3) / 1e12, 1),
        "roofline": {"bound": "mfma", "kernel": dom, "achieved": round(achieved, 1), "peak": peak,
                     "unit": "TFLOP/s", "frac": round(achieved / peak, 4), "traffic": None},
        "kernels": kt, "cpu_baseline": None,
    }
    print(json.dumps(res), flush=True)


def main():
    args = parse()
    if args.gpus != 1:
        print(f"bench.py runs on one GPU only (asked for {args.gpus}): the library has no "
              "multi-GPU path (no collectives or sharding across GPUs).", file=sys.stderr)
        sys.exit(2)
    if args.memory_sweep:
        memory_sweep(args.dw_group_tokens)
        return
    if args.torch_baselines:
        torch_baselines()
        return
    if args.topk:
        bench_topk(args)
        return
    import torch

    import output_head_kl_amd as kd
    import synth

    overrides = {} if args.N is None else {"N": args.N}
    if args.chunk is not None:
        overrides["chunk"] = args.chunk
    t_gen = time.perf_counter()
    inp = synth.make(args.config, **overrides)
    cfg = inp.cfg
    print(f"[bench] generated workload {cfg.name} N={cfg.N} d={cfg.d} V={cfg.V} K={cfg.K} "
          f"chunk={cfg.chunk} in {time.perf_counter() - t_gen:.1f} s", file=sys.stderr, flush=True)
    dev = "cuda"
    if cfg.dtype == "bf16":
        h = torch.from_numpy(inp.h.view(np.int16)).to(dev).view(torch.bfloat16)
        W = torch.from_numpy(inp.W.view(np.int16)).to(dev).view(torch.bfloat16)
    else:
        h, W = torch.from_numpy(inp.h).to(dev), torch.from_numpy(inp.W).to(dev)
    idx = torch.from_numpy(inp.idx).to(dev)
    p = torch.from_numpy(inp.p).to(dev)
    mask = torch.from_numpy(inp.mask).to(dev)
    dt_code = kd.KD_BF16 if cfg.dtype == "bf16" else kd.KD_F32
    ws = torch.empty(kd.workspace_bytes(cfg.N, cfg.d, cfg.V, cfg.K, cfg.chunk, dt_code,
                                        args.dw_group_tokens),
                     dtype=torch.uint8, device=dev)
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()

    def step():
        return kd.fwd_bwd(h, W, idx, p, mask, chunk=cfg.chunk, workspace=ws)

    if args.split:
        return bench_split(args, kd, torch, cfg, h, W, idx, p, mask, ws)
    if args.autograd:
        del ws
        return bench_autograd(args, kd, torch, cfg, h, W, idx, p, mask)
    if args.shard:
        return bench_shard(args, kd, torch, cfg, h, W, idx, p, mask)

    warm_up(step, args.warmup)
    print("[bench] warmup done", file=sys.stderr, flush=True)

    prof = not args.no_profile
    # the clock figure is secondary: a failure to take it leaves it null, never the line
    stamps = torch.zeros((2, 3 * CLOCK_GROUPS), dtype=torch.int64, device=dev)
    clock_err = None
    try:
        kd.clock_stamp(stamps[0])
    except Exception as e:  # noqa: BLE001
        clock_err = f"{type(e).__name__}: {e}"
    with ClockSampler() as clk:
        step_ms, out = timed_steps(step, args.steps)
    clock = None
    try:
        if clock_err is None:
            kd.clock_stamp(stamps[1])
            mhz = unit_clocks(stamps[0].cpu().numpy(), stamps[1].cpu().numpy(),
                              kd.wall_clock_khz())
            if mhz.size:
                clock = {
                    "gfx_mhz_median": round(float(np.median(mhz)), 1),
                    "gfx_mhz_min": round(float(mhz.min()), 1),
                    "gfx_mhz_max": round(float(mhz.max()), 1),
                    "compute_units": int(mhz.size),
                    "source": "each compute unit's shader cycle counter against the constant-rate "
                              "counter, stamped by kd_clock_stamp right before and after the "
                              "timed steps"}
    except Exception as e:  # noqa: BLE001
        clock_err = f"{type(e).__name__}: {e}"
    if clock is None and clock_err:
        print(f"[bench] no measured clock: {clock_err}", file=sys.stderr, flush=True)
    loss_val = float(out[0].item())
    del out
    ms_profiled = None
    if prof:
        # Per-kernel times: the same K steps again with HIP events recorded on the
        # library's stream around every launch (after recorded steps for at least 0.5 s,
        # discarded).  The records cost ~1 ms per step, so they stay out of the pass that
        # gives `value`.
        kd.profile_read()          # discard anything recorded so far
        kd.profile_enable(True)
        warm_up(step, 1)           # recorded and discarded (event pool, steady clock)
        kd.profile_read()
        tp = time.perf_counter()
        for _ in range(args.steps):
            out = None
            out = step()
        torch.cuda.synchronize()
        ms_profiled = (time.perf_counter() - tp) / args.steps * 1e3
        kd.profile_enable(False)
        ktimes = kd.profile_read()
        del out
    peak_gib = torch.cuda.max_memory_allocated() / 2**30

    ms = float(np.median(step_ms))
    tokens_per_s = cfg.N / (ms * 1e-3)
    # the fused call runs three GEMMs per chunk (z, dh, dW): its backward takes dz from the
    # forward's exp(z - max) instead of recomputing z, so 6NVd flops are executed; 8NVd is
    # the work of the recompute formulation (the split fwd/bwd entry points), for context
    flops_step = 6.0 * cfg.N * cfg.V * cfg.d
    tflops = flops_step / (ms * 1e-3) / 1e12
    tflops_recompute_equiv = 8.0 * cfg.N * cfg.V * cfg.d / (ms * 1e-3) / 1e12
    peak = PEAK_BF16_TFLOPS if cfg.dtype == "bf16" else PEAK_F32_TFLOPS
    workload = f"fused_kl_fwd_bwd_N{cfg.N}_d{cfg.d}_V{cfg.V}_K{cfg.K}_chunk{cfg.chunk}_{cfg.dtype}"
    if args.dw_group_tokens is not None:
        workload += f"_dwgroup{args.dw_group_tokens}"

    roofline = None
    kernels = {}
    if prof:
        for name, (tot, n) in ktimes.items():
            if n:
                kernels[name] = {"total_ms_per_step": tot / args.steps, "launches_per_step": n / args.steps,
                                 "avg_ms": tot / n}
        gem = {k: v for k, v in kernels.items() if k in GEMM_CLASSES}
        if gem:
            dom = max(gem, key=lambda k: gem[k]["total_ms_per_step"])
            # every GEMM launch processes one chunk: 2 * rows * V * d flops (rows = chunk
            # except for a partial last chunk, averaged here over the step)
            flops_launch = 2.0 * cfg.N * cfg.V * cfg.d / gem[dom]["launches_per_step"]
            achieved = flops_launch / (gem[dom]["avg_ms"] * 1e-3) / 1e12
            roofline = {"bound": "mfma", "kernel": dom, "achieved": round(achieved, 1),
                        "peak": peak, "unit": "TFLOP/s", "frac": round(achieved / peak, 4),
                        "traffic": traffic_for(dom, workload)}

    headline = (cfg.N, cfg.d, cfg.V, cfg.K) == (32768, 3072, 128256, 100)
    res = {
        "metric": ("tokens/s + MFMA util, fused KL fwd+bwd, N=32K d=3072 V=128256 K=100"
                   if headline else f"tokens/s + MFMA util, fused KL fwd+bwd, N={cfg.N} "
                                    f"d={cfg.d} V={cfg.V} K={cfg.K}"),
        "value": round(tokens_per_s, 1),
        "unit": "tokens/s",
        "n_gpus": 1,
        "steps": args.steps,
        "warmup": args.warmup,
        "ms_per_step": round(ms, 3),
        "ms_per_step_mean": round(float(np.mean(step_ms)), 3),
        "ms_per_step_all": [round(x, 3) for x in step_ms],
        "higher_is_better": True,
        "scaling": "weak",
        "vs_baseline": None,
        "dtype": cfg.dtype,
        "data": "synthetic",
        "config": {"workload": workload, "N": cfg.N, "d": cfg.d, "V": cfg.V, "K": cfg.K,
                   "chunk": cfg.chunk, "mask": cfg.mask,
                   "dw_group_tokens": 16384 if args.dw_group_tokens is None else args.dw_group_tokens},
        "workspace_bytes": ws.numel(),
        "tflops_executed_6NVd": round(tflops, 1),
        "frac_of_peak_executed": round(tflops / peak, 4),
        "tflops_recompute_equiv_8NVd": round(tflops_recompute_equiv, 1),
        # the peak assumes 2.4 GHz; against the clock the chip actually ran at
        "clock_observed": clock,
        "frac_of_peak_at_observed_clock": (
            None if clock is None else round(tflops / (peak * clock["gfx_mhz_median"] / 2400.0), 4)),
        "clock_amdsmi": clk.result(),
        "peak_mem_gib": round(peak_gib, 3),
        "loss": loss_val,
        "roofline": roofline,
        "kernels": kernels,
        "ms_per_step_profiled_pass": None if ms_profiled is None else round(ms_profiled, 3),
        "cpu_baseline": None,
    }
    if args.dw_group_tokens is None and not args.no_small_workspace and cfg.dtype == "bf16":
        # the same workload with the smallest workspace the call accepts: dW is accumulated
        # chunk by chunk, so no buffer holds more than one chunk of logits
        del ws
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        ws0 = torch.empty(kd.workspace_bytes(cfg.N, cfg.d, cfg.V, cfg.K, cfg.chunk, dt_code, 0),
                          dtype=torch.uint8, device=dev)
        torch.cuda.synchronize()
        torch.cuda.reset_peak_memory_stats()

        def step0():
            return kd.fwd_bwd(h, W, idx, p, mask, chunk=cfg.chunk, workspace=ws0)

        warm_up(step0, 1)
        t0_ms, out0 = timed_steps(step0, args.steps)
        res["smallest_workspace"] = {
            "dw_group_tokens": 0, "workspace_bytes": ws0.numel(),
            "ms_per_step": round(float(np.median(t0_ms)), 3),
            "tokens_per_s": round(cfg.N / (float(np.median(t0_ms)) * 1e-3), 1),
            "peak_mem_gib": round(torch.cuda.max_memory_allocated() / 2**30, 3),
            "loss": float(out0[0].item())}
        del out0, ws0
    if (cfg.dtype == "bf16" and roofline is not None and roofline["kernel"] == "fwd_gemm_lse"
            and not args.no_reference):
        try:  # context only: a failure here leaves the line whole
            res["gemm_reference"] = gemm_reference(torch, h, W, cfg,
                                                   kernels["fwd_gemm_lse"]["avg_ms"])
        except Exception as e:  # noqa: BLE001
            res["gemm_reference"] = {"error": f"{type(e).__name__}: {e}"}
    if args.copy_gib > 0:
        n = int(args.copy_gib * 2**30) // 4
        src = torch.ones(n, dtype=torch.float32, device=dev)
        dst = torch.empty_like(src)
        torch.cuda.synchronize()
        dst.copy_(src)
        torch.cuda.synchronize()
        res["copy_bytes_each_way"] = n * 4
        del src, dst
    if not args.no_cpu_baseline:
        print("[bench] timing the CPU oracle", file=sys.stderr, flush=True)
        res["cpu_baseline"] = cpu_baseline(inp, args.cpu_rows)
    print(json.dumps(res), flush=True)


if __name__ == "__main__":
    main()
