"""Bench: batched prompt-lookup drafting on one MI355X.

A step is one pld_draft_batch call over the whole batch (scan + gather, one
kernel) on the 16 x 262,144-token workload (Zipf(1.1) documents with a
4,096-token copied tail, 0.5% substitutions; n 4..12, k_max 16). Inputs are
resident in HBM when timing starts.

Steps run from HIP graphs of up to --graph-steps captured calls: exactly
--warmup untimed steps, then exactly --steps timed steps (n steps are n // G
replays of a G-step graph and one replay of an (n % G)-step graph). Each
captured graph is replayed once beforehand and compared with an eager call.

Reported (one JSON line on stdout):
  value         draft steps/s: host clock around the K timed steps, with a
                device synchronize on each side. Each step reads a different
                one of R copies of the batch (R * 16.8 MB >= 512 MB), so the
                256 MB Infinity Cache cannot serve repeats.
  scan_GBps     4 * sum(L) bytes / the kernel's mean launch time, taken with
                HIP events on the launch stream around the same K steps (one
                kernel per step).
  roofline      the same against MI355X's 8 TB/s HBM peak; `traffic` is the
                HBM bytes per launch from the committed rocprofv3 counter
                summary, used only while the profiled sources still match it.
  p50_us/p90_us latency of one call: HIP event pair around a single eager
                call (this includes the event-pair overhead of the runtime);
                p50_GBps the history bytes over that median.
  cpu_baseline  the CPU oracle on the same batch, one thread; and, for
                context, cpu_baseline_threads: the same oracle one request per
                task over the host cores.
"""

from __future__ import annotations

import argparse
import json
import os
import platform
import sys
import time

import numpy as np

ROOT = os.path.dirname(os.path.abspath(__file__))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

METRIC = ("batched draft steps/s + scanned history GB/s (% HBM peak); "
          "p50 µs per draft step")
METRIC_NGRAM = ("successor-count n-gram draft steps/s (llama.cpp context cache rule, "
                "batched, exact)")
METRIC_FUSE = ("lookup draft + draft fusion and long-block scheduling steps/s "
               "(HyperQwen lookup-drafting page, steps 1-3)")
# counter summaries of pld_scan per lookup workload (default launch), and of
# the one-launch lookup + fusion step
PROFILES = {1: "pld_scan_c1_b1x4096.md", 2: "pld_scan_c2_b8x25000.md",
            3: "pld_scan_c3_b64_ragged.md", 4: "pld_scan_c4_b16x262144.md"}
PROFILES_FUSE = {4: "pld_scan_fused_c4_b16x262144.md"}
PROFILE_APPEND_DRAFT = "pld_scan_append_c5_stream_b64.md"
PROFILE_STREAM = "pld_scan_c5_stream_b64.md"
# the sources a counter summary is valid for: the kernels, the C-ABI layer
# that picks their launch (tile, grid) and the build script that sets their
# compiler flags
CSRC = os.path.join(ROOT, "prompt_lookup_gram_amd", "csrc")
PROFILED_SOURCES = ("pld_kernels.hip", "pld_kernels.h", "pld_device.h", "pld_api.cpp",
                    os.path.join(os.pardir, "build.py"))
TIME_SOURCE = ("value, ms_per_step: host clock around the K timed steps, with a device "
               "synchronize on each side; graph_us_per_step, scan_GBps and roofline: HIP "
               "events recorded on the launch stream around the same K steps")


def source_hash() -> str:
    """First 16 hex digits of the SHA-256 of the profiled sources, in order."""
    import hashlib
    h = hashlib.sha256()
    for name in PROFILED_SOURCES:
        with open(os.path.join(CSRC, name), "rb") as f:
            h.update(f.read())
    return h.hexdigest()[:16]


def calibration_copies(torch, dev):
    """8 device copies of a 64 MiB int32 tensor: a kernel of known size whose
    FETCH_SIZE / WRITE_SIZE scale the counter profiles."""
    src = torch.randint(0, 1 << 30, (16 << 20,), dtype=torch.int32, device=dev)
    dst = torch.empty_like(src)
    for _ in range(8):
        dst.copy_(src)
    torch.cuda.synchronize()


def profiled_traffic(name, key="traffic-bytes-per-launch"):
    """HBM bytes per launch from a committed counter summary, if it was taken
    on the sources as they are now (else None). The default key is the
    FETCH_SIZE + WRITE_SIZE figure scaled by a plain copy's reading;
    "traffic-sized-bytes-per-launch" counts the read requests by size."""
    if name is None:
        return None
    try:
        text = open(os.path.join(ROOT, "profiles", name)).read()
        src = source_hash()
    except OSError:
        return None
    sha = traffic = None
    for line in text.splitlines():
        if line.startswith("source-sha256-16:"):
            sha = line.split(":", 1)[1].strip()
        if line.startswith(key + ":"):
            traffic = int(line.split(":", 1)[1].strip())
    return traffic if sha == src else None


TRAFFIC_NOTE = ("traffic: FETCH_SIZE and WRITE_SIZE per launch, each scaled by its reading "
                "for a 64 MiB copy; traffic_by_request_size: the L2's 128-, 64- and 32-byte "
                "read requests counted at their sizes, plus WRITE_SIZE (both from the "
                "committed counter summary of this workload, used while the profiled "
                "sources match it)")


def step_plan(n: int, g: int) -> list:
    """Graph sizes whose replays run exactly n steps: n // g replays of a
    g-step graph, then one replay of an (n % g)-step graph."""
    q, r = divmod(max(0, int(n)), int(g))
    return [g] * q + ([r] if r else [])


class GraphSteps:
    """Steps replayed from HIP graphs captured on a side stream. capture(m)
    records steps 0..m-1; it is called once for each graph size in use."""

    def __init__(self, torch, capture, g):
        self.torch, self.capture, self.g = torch, capture, int(g)
        self.graphs = {}
        self.stream = torch.cuda.Stream()

    def prepare(self, *counts):
        """Capture every graph that running each of `counts` steps needs;
        returns the captured sizes."""
        torch = self.torch
        for n in counts:
            for m in step_plan(n, self.g):
                if m not in self.graphs:
                    graph = torch.cuda.CUDAGraph()
                    torch.cuda.synchronize()
                    with torch.cuda.graph(graph, stream=self.stream):
                        self.capture(m)
                    torch.cuda.synchronize()
                    self.graphs[m] = graph
        return sorted(self.graphs)

    def run(self, n):
        for m in step_plan(n, self.g):
            self.graphs[m].replay()

    def last(self, n):
        """Size of the graph that runs the last of n steps."""
        plan = step_plan(n, self.g)
        return plan[-1] if plan else 0


def timed_steps(torch, gs, k):
    """Exactly k steps between two device synchronizes: (host seconds, HIP
    event seconds on the current stream, where the graphs are launched)."""
    e0 = torch.cuda.Event(enable_timing=True)
    e1 = torch.cuda.Event(enable_timing=True)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    e0.record()
    gs.run(k)
    e1.record()
    torch.cuda.synchronize()
    return time.perf_counter() - t0, e0.elapsed_time(e1) * 1e-3


HBM_PEAK_GBPS = 8000.0
MALL_BYTES = 256 * 2 ** 20


def parse():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--gpus", type=int, default=1)
    ap.add_argument("--steps", type=int, default=4096)
    ap.add_argument("--warmup", type=int, default=256)
    ap.add_argument("--config", type=int, default=4, choices=[1, 2, 3, 4, 5],
                    help="workload: 4 (default) is the 16 x 262,144 batch; 1-3 "
                         "the smaller batches; 5 the 1,024-step streaming decode")
    ap.add_argument("--layout", choices=["strided", "rows"], default="rows",
                    help="histories through a row-pointer table (pld_draft_batch, "
                         "the default) or as one padded [batch, stride] buffer per "
                         "copy (pld_draft_batch_strided, min_len = the shortest "
                         "history)")
    ap.add_argument("--graph-steps", type=int, default=128,
                    help="draft calls captured per HIP graph")
    ap.add_argument("--latency-calls", type=int, default=200)
    ap.add_argument("--tile", type=int, default=0, help="0 = library default")
    ap.add_argument("--fused", type=int, default=-1, help="-1 = library default")
    ap.add_argument("--cpu-seconds", type=float, default=10.0)
    ap.add_argument("--no-cpu-baseline", action="store_true")
    ap.add_argument("--warm", action="store_true",
                    help="also time without buffer rotation (cache-resident)")
    ap.add_argument("--fuse", choices=["none", "one", "two"], default="none",
                    help="each step also fuses the lookup draft with a drafter's "
                         "proposal and schedules the block (one launch: "
                         "pld_draft_fuse_batch; two: pld_draft_batch + pld_fuse); "
                         "row-table layout, workloads 1-4")
    ap.add_argument("--ngram", action="store_true",
                    help="draft from the successor-count cache (pld_create_ngram, "
                         "pld_draft_ngram) instead of the lookup scan")
    ap.add_argument("--index", action="store_true",
                    help="workload 5 only: draft from the context's incremental n-gram "
                         "index (pld_create_indexed, pld_draft_store) instead of scanning")
    ap.add_argument("--stream-start", type=int, default=0,
                    help="workload 5 only: start histories of this many tokens instead "
                         "of 32,768 (the same decode on longer histories)")
    ap.add_argument("--control", action="store_true",
                    help="workload 5 only: each step also runs the online cost/benefit "
                         "controller (pld_control) on the step's lookup drafts")
    ap.add_argument("--control-fused", action="store_true",
                    help="workload 5, scan drafting: the controller step runs in the draft's "
                         "own launch (pld_draft_control_batch)")
    ap.add_argument("--append-draft", action="store_true",
                    help="workload 5 only: each step's append and the next step's draft "
                         "as one pld_append_draft_store call")
    ap.add_argument("--verify-step", action="store_true",
                    help="workload 5's start histories: time one verify step (the lookup "
                         "draft, the block's keys and values into a paged cache, attention "
                         "of the block, verification of the draft) instead of the drafting")
    ap.add_argument("--library-read", action="store_true",
                    help="also time torch.amax over the same rotated copies (a library "
                         "full read of the same bytes, for context)")
    ap.add_argument("--calibrate-copy", action="store_true",
                    help="finish with 8 plain 64 MiB device copies (a counter "
                         "reference of known size for rocprofv3 --pmc)")
    ap.add_argument("--print-source-hash", action="store_true",
                    help="print the hash a counter summary under profiles/ records for "
                         "the kernel sources, and exit")
    return ap.parse_args()


def cpu_model() -> str:
    try:
        for line in open("/proc/cpuinfo"):
            if line.startswith("model name"):
                return line.split(":", 1)[1].strip()
    except OSError:
        pass
    return platform.processor() or "unknown"


def main():
    args = parse()
    if args.print_source_hash:
        print(source_hash())
        return
    if args.steps < 1 or args.warmup < 0:
        print("--steps must be at least 1 and --warmup at least 0", file=sys.stderr)
        sys.exit(2)
    world = int(os.environ.get("WORLD_SIZE", "1"))
    if args.gpus != 1 or world != 1:
        print("bench.py runs on exactly one GPU: requests shard across GPUs with "
              "no exchange, so the per-GPU figure is the whole story; "
              f"--gpus {args.gpus} (WORLD_SIZE={world}) is not supported.",
              file=sys.stderr)
        sys.exit(2)

    import torch

    from prompt_lookup_gram_amd import binding as B
    from prompt_lookup_gram_amd import workloads as wl

    assert torch.cuda.is_available(), "bench.py needs a GPU"
    torch.cuda.set_device(0)
    dev = torch.device("cuda:0")
    B.load()

    if args.control_fused:
        args.control = True
        if args.index or args.ngram or args.append_draft or args.config != 5:
            print("--control-fused: workload 5 with scan drafting only (pld_draft_control_batch)",
                  file=sys.stderr)
            sys.exit(2)
    if args.ngram and (args.index or args.fuse != "none"):
        print("--ngram drafts from the successor-count cache: it does not combine with "
              "--index or --fuse", file=sys.stderr)
        sys.exit(2)
    if args.verify_step:
        if args.config != 5 or args.index or args.ngram or args.fuse != "none" or args.control \
                or args.append_draft:
            print("--verify-step: workload 5 with scan drafting only", file=sys.stderr)
            sys.exit(2)
        return bench_verify_step(args, torch, B, wl, dev)
    if args.config == 5:
        return bench_stream(args, torch, B, wl, dev)

    w = wl.ALL_CONFIGS[args.config]()
    if args.ngram:
        return bench_ngram(args, torch, B, wl, dev, w)
    if args.fuse != "none":
        return bench_fuse(args, torch, B, wl, dev, w)
    bytes_step = 4 * w.total_tokens
    # enough copies to defeat the Infinity Cache, capped for the tiny batches
    # (which are launch-latency bound either way)
    rot = min(64, max(1, -(-2 * MALL_BYTES // bytes_step)))
    out = B.alloc_outputs(w.batch, w.k_max, device=dev)
    if args.layout == "strided":
        sb = B.StridedBatch(w.histories, device=dev)
        bufs = [sb.buf] + [sb.buf.clone() for _ in range(rot - 1)]
        ctx = B.pld_create(w.batch, sb.max_len)

        def call(i, stream=None):
            B.pld_draft_batch_strided(ctx, bufs[i % rot], sb.stride, sb.lengths, sb.min_len,
                                      w.batch, w.n_min, w.n_max, w.k_max, out[0], out[1],
                                      out[2], stream=stream)
    else:
        base = B.DeviceBatch(w.histories, device=dev)
        copies = [base] + [base.replicate() for _ in range(rot - 1)]
        # the row-pointer tables of all copies share one small allocation, as
        # a serving loop's per-request metadata would; only the histories rotate
        rows_all = torch.stack([c.rows for c in copies]).contiguous()
        ctx = B.pld_create(w.batch, base.max_len)

        def call(i, stream=None):
            r = i % rot
            B.pld_draft_batch(ctx, rows_all[r], copies[r].lengths, w.batch, w.n_min,
                              w.n_max, w.k_max, out[0], out[1], out[2], stream=stream)
    B.pld_configure(ctx, args.tile, args.fused)
    tile = B.pld_scan_tile(ctx, w.batch)   # the tile the library launches

    # reference output (eager) for the graph check and the parity check
    call(0)
    assert B.pld_sync(ctx) == B.PLD_OK
    eager = [t.clone() for t in out[:3]]

    # ---- HIP graphs of consecutive steps (rotating copies) ------------------
    G = max(1, min(args.graph_steps, args.steps))
    gs = GraphSteps(torch, lambda m: [call(i) for i in range(m)], G)

    def check_out(what):
        for a_, b_ in zip(eager, out[:3]):
            assert torch.equal(a_, b_), f"{what} differs from the eager call"

    graph_sizes = gs.prepare(args.steps, args.warmup)
    for m in graph_sizes:  # each captured graph reproduces the eager result
        for t in out[:3]:
            t.fill_(-9)
        gs.graphs[m].replay()
        torch.cuda.synchronize()
        check_out(f"a replay of the {m}-step graph")
    gs.run(args.warmup)                     # exactly W untimed steps
    wall_s, gpu_s = timed_steps(torch, gs, args.steps)   # exactly K timed steps
    check_out("the last timed step")
    steps = args.steps
    gpu_ms = gpu_s * 1e3
    ms_per_step = wall_s * 1e3 / steps
    steps_per_s = steps / wall_s

    # ---- per-call latency and kernel time: event pairs around eager calls ---
    n_lat = max(10, args.latency_calls)
    s = torch.cuda.current_stream()
    starts = [torch.cuda.Event(enable_timing=True) for _ in range(n_lat)]
    ends = [torch.cuda.Event(enable_timing=True) for _ in range(n_lat)]
    for i in range(64):
        call(i)
    torch.cuda.synchronize()
    for i in range(n_lat):
        starts[i].record(s)
        call(i)
        ends[i].record(s)
    torch.cuda.synchronize()
    lat_us = np.array([a.elapsed_time(b_) * 1e3 for a, b_ in zip(starts, ends)])
    p50, p90, mean_us = (float(np.percentile(lat_us, 50)),
                         float(np.percentile(lat_us, 90)), float(lat_us.mean()))

    warm = None
    if args.warm:
        g2 = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g2, stream=gs.stream):
            for i in range(G):
                call(0)
        torch.cuda.synchronize()
        g2.replay()
        torch.cuda.synchronize()
        reps = max(1, steps // G)
        e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        e0.record()
        for _ in range(reps):
            g2.replay()
        e1.record()
        torch.cuda.synchronize()
        warm_us = e0.elapsed_time(e1) * 1e3 / (reps * G)
        warm = {"us_per_step": warm_us, "GBps": bytes_step / warm_us / 1e3,
                "note": "same copy every step (Infinity-Cache resident)"}

    library = None
    if args.library_read:
        # torch's own full reduction over each rotated copy, graph-replayed
        flat = [b.reshape(-1) for b in (bufs if args.layout == "strided" else
                                         [c.flat for c in copies])]
        red = torch.empty((), dtype=torch.int32, device=dev)
        g3 = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g3, stream=gs.stream):
            for i in range(G):
                torch.amax(flat[i % rot], 0, out=red)
        torch.cuda.synchronize()
        g3.replay()
        torch.cuda.synchronize()
        reps = max(1, steps // G)
        e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        e0.record()
        for _ in range(reps):
            g3.replay()
        e1.record()
        torch.cuda.synchronize()
        lib_us = e0.elapsed_time(e1) * 1e3 / (reps * G)
        library = {"op": "torch.amax over the same rotated copies", "us_per_launch": lib_us,
                   "GBps": flat[0].numel() * 4 / lib_us / 1e3}

    assert B.pld_sync(ctx) == B.PLD_OK
    got = [t.cpu().numpy() for t in out[:3]]
    B.pld_destroy(ctx)

    if args.calibrate_copy:
        calibration_copies(torch, dev)

    graph_us = gpu_ms * 1e3 / steps           # mean launch time (one kernel per step)
    scan_gbps = bytes_step / (graph_us * 1e-6) / 1e9
    default_launch = (args.tile in (0, tile) and args.fused in (-1, 1)
                      and args.layout == "rows")
    prof = PROFILES.get(args.config) if default_launch else None
    traffic, traffic_sized = (profiled_traffic(prof),
                              profiled_traffic(prof, "traffic-sized-bytes-per-launch"))
    rec = {
        "metric": METRIC,
        "value": round(steps_per_s, 1),
        "unit": "draft steps/s",
        "n_gpus": 1,
        "steps": steps,
        "warmup": args.warmup,
        "ms_per_step": round(ms_per_step, 6),
        "higher_is_better": True,
        "scaling": "weak",
        "vs_baseline": None,
        "dtype": "int32",
        "data": "synthetic",
        "time_source": TIME_SOURCE,
        "config": {"workload": w.name, "batch": w.batch, "layout": args.layout,
                   "tile_tokens": tile,
                   "history_tokens": int(w.lengths.max()),
                   "n_min": w.n_min, "n_max": w.n_max, "k_max": w.k_max,
                   "bytes_per_step": bytes_step, "rotated_copies": rot,
                   "graph_steps": G, "graph_sizes": graph_sizes},
        "capture_check": "each captured graph replayed once before the warm-up and "
                         "compared with an eager call; the last timed step compared too",
        "request_drafts_per_s": round(steps_per_s * w.batch, 1),
        "scan_GBps": round(scan_gbps, 1),
        "hbm_frac": round(scan_gbps / HBM_PEAK_GBPS, 4),
        "p50_us": round(p50, 3),
        "p90_us": round(p90, 3),
        # the whole eager step at its median latency, launch included
        "p50_GBps": round(bytes_step / (p50 * 1e-6) / 1e9, 1),
        "graph_us_per_step": round(graph_us, 3),
        "eager_call_mean_us": round(mean_us, 3),
        "roofline": {"bound": "hbm", "achieved": round(scan_gbps, 1),
                     "peak": HBM_PEAK_GBPS, "unit": "GB/s",
                     "frac": round(scan_gbps / HBM_PEAK_GBPS, 4), "traffic": traffic,
                     "traffic_by_request_size": traffic_sized, "traffic_note": TRAFFIC_NOTE,
                     "kernel": "pld_scan",
                     "time_source": "HIP events on the launch stream around the K "
                                    f"timed steps ({steps} launches, rotated copies)"},
    }
    if warm:
        rec["warm"] = warm
    if library:
        rec["library_full_read"] = library

    if not args.no_cpu_baseline:
        import oracle
        od, ol, om, _ = oracle.draft(w.histories, w.n_min, w.n_max, w.k_max)
        parity = (np.array_equal(got[0], od) and np.array_equal(got[1], ol)
                  and np.array_equal(got[2], om))
        n, t_start = 0, time.perf_counter()
        while True:
            oracle.draft(w.histories, w.n_min, w.n_max, w.k_max)
            n += 1
            el = time.perf_counter() - t_start
            if el >= args.cpu_seconds:
                break
        rec["cpu_baseline"] = {
            "value": round(n / el, 3), "unit": "draft steps/s", "cores": 1,
            "kind": "oracle",
            "sample": f"{n} full steps of the same {w.batch}-request batch "
                      f"({el:.1f} s, one thread, {cpu_model()}, "
                      f"{len(os.sched_getaffinity(0))} host cores visible)",
            "effective_GBps": round(bytes_step * n / el / 1e9, 3),
        }
        # secondary, for context: the same oracle fanned out one request per
        # task over the host cores (its C call releases the GIL)
        from concurrent.futures import ThreadPoolExecutor
        cores = len(os.sched_getaffinity(0))

        def one(h):
            oracle.draft([h], w.n_min, w.n_max, w.k_max)

        with ThreadPoolExecutor(max_workers=cores) as ex:
            n2, t2 = 0, time.perf_counter()
            while True:
                list(ex.map(one, w.histories))
                n2 += 1
                el2 = time.perf_counter() - t2
                if el2 >= args.cpu_seconds / 2:
                    break
        rec["cpu_baseline_threads"] = {
            "value": round(n2 / el2, 3), "unit": "draft steps/s",
            "cores": min(cores, w.batch), "kind": "oracle",
            "sample": f"{n2} full steps of the same batch, one request per task on a pool of "
                      f"{cores} threads ({el2:.1f} s, {cpu_model()})",
        }
        rec["parity"] = "bit-exact" if parity else "MISMATCH"
        if not parity:
            print(json.dumps(rec))
            sys.exit(1)
    print(json.dumps(rec), flush=True)


def bench_fuse(args, torch, B, wl, dev, w):
    """Lookup drafting plus draft fusion and long-block scheduling per step.

    Each step drafts the batch (rotated copies, as the plain bench) and fuses
    the drafts with a drafter's 7-token proposal under the page's parameters,
    the schedule state carried on the device. Drafter proposals are seeded
    draws; each step's accepted count is drawn against the previous block's
    positions in one untimed eager pass (mostly near-full, as while copying),
    so the graph of G steps (state zeroed first) replays exactly that pass.
    """
    import torch as _t
    bytes_step = 4 * w.total_tokens
    rot = min(64, max(1, -(-2 * MALL_BYTES // bytes_step)))
    G = max(1, min(args.graph_steps, args.steps))
    k = w.k_max
    params = B.pld_fuse_params_default()
    n_pos = params.positions_long
    base = B.DeviceBatch(w.histories, device=dev)
    copies = [base] + [base.replicate() for _ in range(rot - 1)]
    rows_all = _t.stack([c.rows for c in copies]).contiguous()
    ctx = B.pld_create(w.batch, base.max_len)
    B.pld_configure(ctx, args.tile, args.fused)
    tile = B.pld_scan_tile(ctx, w.batch)
    default_launch = args.tile in (0, tile) and args.fused in (-1, 1) and args.fuse == "one"
    prof = PROFILES_FUSE.get(args.config) if default_launch else None
    traffic, traffic_sized = (profiled_traffic(prof),
                              profiled_traffic(prof, "traffic-sized-bytes-per-launch"))
    out = B.alloc_outputs(w.batch, k, device=dev)
    state = _t.zeros((w.batch, B.PLD_FUSE_STATE_WORDS), dtype=_t.int32, device=dev)
    blk = _t.empty((w.batch, n_pos), dtype=_t.int32, device=dev)
    pos = _t.empty(w.batch, dtype=_t.int32, device=dev)
    src = _t.empty(w.batch, dtype=_t.int64, device=dev)
    rng = np.random.default_rng([8001, args.config])
    drafter = rng.integers(0, wl.ZIPF_VOCAB, size=(G, w.batch, params.head)).astype(np.int32)
    drafter_d = _t.from_numpy(drafter).to(dev)
    acc = np.zeros((G, w.batch), np.int32)
    acc_d = _t.zeros((G, w.batch), dtype=_t.int32, device=dev)

    def call(i, stream=None):
        r = i % rot
        if args.fuse == "one":
            B.pld_draft_fuse_batch(ctx, rows_all[r], copies[r].lengths, w.batch, w.n_min,
                                   w.n_max, k, out[0], out[1], out[2], params, drafter_d[i % G],
                                   acc_d[i % G], state, blk, pos, src, stream=stream)
        else:
            B.pld_draft_batch(ctx, rows_all[r], copies[r].lengths, w.batch, w.n_min, w.n_max,
                              k, out[0], out[1], out[2], stream=stream)
            B.pld_fuse(ctx, params, out[0], k, out[1], out[2], drafter_d[i % G], acc_d[i % G],
                       state, w.batch, blk, pos, src, stream=stream)

    # untimed eager pass: fixes each step's accepted count
    trace = []
    for i in range(G):
        acc_d[i].copy_(_t.from_numpy(acc[i]))
        call(i)
        p_ = pos.cpu().numpy()
        trace.append((out[0].cpu().numpy(), out[1].cpu().numpy(), out[2].cpu().numpy(),
                      blk.cpu().numpy(), p_, src.cpu().numpy(), state.cpu().numpy()))
        if i + 1 < G:
            short = rng.choice([0, 0, 0, 1, 1, 2, 4, 7], size=w.batch)
            acc[i + 1] = np.maximum(p_ - short, 0)
    assert B.pld_sync(ctx) == B.PLD_OK
    long_frac = float(np.mean([t[6][:, 0] for t in trace]))
    mean_pos = float(np.mean([t[4] for t in trace]))

    def capture(m):  # schedule state zeroed, then steps 0..m-1 of the eager pass
        state.zero_()
        for i in range(m):
            call(i)

    gs = GraphSteps(_t, capture, G)

    def check_step(m, what):  # the state after m steps from zero
        assert np.array_equal(blk.cpu().numpy(), trace[m - 1][3]), what
        assert np.array_equal(state.cpu().numpy(), trace[m - 1][6]), what

    graph_sizes = gs.prepare(args.steps, args.warmup)
    for m in graph_sizes:  # each captured graph reproduces the eager pass
        blk.fill_(-9)
        gs.graphs[m].replay()
        _t.cuda.synchronize()
        check_step(m, f"a replay of the {m}-step graph differs from the eager pass")
    gs.run(args.warmup)
    wall_s, gpu_s = timed_steps(_t, gs, args.steps)
    check_step(gs.last(args.steps), "the last timed step differs from the eager pass")
    steps = args.steps
    gpu_us = gpu_s * 1e6 / steps
    assert B.pld_sync(ctx) == B.PLD_OK
    B.pld_destroy(ctx)
    if args.calibrate_copy:
        calibration_copies(_t, dev)
    scan_gbps = bytes_step / (gpu_us * 1e-6) / 1e9
    launches = 1 if args.fuse == "one" else 2
    rec = {
        "metric": METRIC_FUSE,
        "value": round(steps / wall_s, 1),
        "unit": "draft+fuse steps/s",
        "n_gpus": 1,
        "steps": steps,
        "warmup": args.warmup,
        "ms_per_step": round(wall_s * 1e3 / steps, 6),
        "higher_is_better": True,
        "scaling": "weak",
        "vs_baseline": None,
        "dtype": "int32",
        "data": "synthetic",
        "time_source": TIME_SOURCE,
        "config": {"workload": w.name, "batch": w.batch, "layout": "rows",
                   "history_tokens": int(w.lengths.max()), "n_min": w.n_min,
                   "n_max": w.n_max, "k_max": k, "bytes_per_step": bytes_step,
                   "rotated_copies": rot, "graph_steps": G, "graph_sizes": graph_sizes,
                   "tile_tokens": tile,
                   "fuse": {f: getattr(params, f) for f, _ in params._fields_},
                   "launches_per_step": launches},
        "capture_check": "each captured graph (schedule state zeroed first) replayed once "
                         "before the warm-up and compared with the eager pass; the last "
                         "timed step compared too",
        "graph_us_per_step": round(gpu_us, 3),
        "scan_GBps": round(scan_gbps, 1),
        "hbm_frac": round(scan_gbps / HBM_PEAK_GBPS, 4),
        "long_block_step_frac": round(long_frac, 4),
        "mean_draft_positions": round(mean_pos, 3),
        # one launch per step: the step's time is the kernel's own; two: the
        # whole step, a lower bound of the scan kernel's fraction
        "roofline": {"bound": "hbm", "achieved": round(scan_gbps, 1), "peak": HBM_PEAK_GBPS,
                     "unit": "GB/s", "frac": round(scan_gbps / HBM_PEAK_GBPS, 4),
                     "traffic": traffic, "traffic_by_request_size": traffic_sized,
                     "traffic_note": TRAFFIC_NOTE,
                     "kernel": ("pld_scan (lookup, fusion and schedule in one launch)"
                                if launches == 1 else "pld_scan + pld_fuse_kernel (whole step)"),
                     "bytes": "history bytes per step (the fusion's per-request inputs and "
                              "outputs, under 200 bytes a request, are not counted)",
                     "time_source": f"HIP events on the launch stream around the K timed "
                                    f"steps ({steps} steps, {launches} launch(es) each, "
                                    f"state zeroed once per graph replay)"},
    }
    if not args.no_cpu_baseline:
        import oracle
        op = oracle.FuseParams(*[getattr(params, f) for f, _ in params._fields_])
        ostate = np.zeros((w.batch, B.PLD_FUSE_STATE_WORDS), np.int32)
        n, parity, t_start = 0, True, time.perf_counter()
        while n < G and time.perf_counter() - t_start < args.cpu_seconds:
            od, ol, om, _ = oracle.draft(w.histories, w.n_min, w.n_max, k)
            ob, opos, osrc, ostate = oracle.fuse(op, od, ol, om, drafter[n], acc[n], ostate)
            g = trace[n]
            parity &= all(np.array_equal(a_, b_) for a_, b_ in
                          zip((od, ol, om, ob, opos, osrc.view(np.int64), ostate), g))
            n += 1
        el = time.perf_counter() - t_start
        rec["cpu_baseline"] = {
            "value": round(n / el, 3), "unit": "draft+fuse steps/s", "cores": 1,
            "kind": "oracle",
            "sample": f"the first {n} steps (lookup oracle then fusion oracle, {el:.1f} s, "
                      f"one thread, {cpu_model()})"}
        rec["parity"] = "bit-exact" if parity else "MISMATCH"
        if not parity:
            print(json.dumps(rec))
            sys.exit(1)
    print(json.dumps(rec), flush=True)


def bench_ngram(args, torch, B, wl, dev, w):
    """Successor-count drafting on a lookup workload's histories.

    The cache is built once by appending every history whole (timed on its
    own: the insert rate), then G draft calls over the batch are captured in
    a HIP graph and replayed. Each call drafts from the same cache state, so
    the slots it reads are warm in the caches after the first replay (the
    streaming leg, --config 5 --ngram, appends between drafts)."""
    G = max(1, min(args.graph_steps, args.steps))
    k = w.k_max
    nb = w.batch
    max_len = int(w.lengths.max())
    ctx = B.pld_create_ngram(nb, max_len)
    params = B.pld_ngram_params_default()
    width = max_len
    tok = np.zeros((nb, width), np.int32)
    for b, h in enumerate(w.histories):
        tok[b, :len(h)] = h
    tok_d = torch.from_numpy(tok).to(dev)
    cnt_d = torch.from_numpy(w.lengths.astype(np.int32)).to(dev)
    out_d = torch.empty((nb, k), dtype=torch.int32, device=dev)
    out_l = torch.empty(nb, dtype=torch.int32, device=dev)
    out_v = torch.empty((nb, k), dtype=torch.int32, device=dev)
    torch.cuda.synchronize()
    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    e0.record()
    B.pld_append(ctx, tok_d, width, cnt_d, nb)
    e1.record()
    torch.cuda.synchronize()
    build_s = e0.elapsed_time(e1) * 1e-3
    B.pld_draft_ngram(ctx, params, nb, k, out_d, out_l, out_v)
    assert B.pld_sync(ctx) == B.PLD_OK
    ref = (out_d.cpu().numpy(), out_l.cpu().numpy(), out_v.cpu().numpy())

    def capture(m):
        for _ in range(m):
            B.pld_draft_ngram(ctx, params, nb, k, out_d, out_l, out_v)

    gs = GraphSteps(torch, capture, G)

    def check_out(what):
        assert (np.array_equal(out_d.cpu().numpy(), ref[0])
                and np.array_equal(out_l.cpu().numpy(), ref[1])
                and np.array_equal(out_v.cpu().numpy(), ref[2])), what

    graph_sizes = gs.prepare(args.steps, args.warmup)
    for m in graph_sizes:
        out_d.fill_(-9)
        gs.graphs[m].replay()
        torch.cuda.synchronize()
        check_out(f"a replay of the {m}-step graph differs from the eager call")
    gs.run(args.warmup)
    wall_s, gpu_s = timed_steps(torch, gs, args.steps)
    check_out("the last timed step differs from the eager call")
    steps = args.steps
    gpu_us = gpu_s * 1e6 / steps
    assert B.pld_sync(ctx) == B.PLD_OK
    B.pld_destroy(ctx)
    if args.calibrate_copy:
        calibration_copies(torch, dev)
    rec = {
        "metric": METRIC_NGRAM,
        "value": round(steps / wall_s, 1),
        "unit": "draft steps/s",
        "n_gpus": 1,
        "steps": steps,
        "warmup": args.warmup,
        "ms_per_step": round(wall_s * 1e3 / steps, 6),
        "higher_is_better": True,
        "scaling": "weak",
        "vs_baseline": None,
        "dtype": "int32",
        "data": "synthetic",
        "time_source": TIME_SOURCE.replace("scan_GBps and roofline", "ns_per_drafted_token"),
        "config": {"workload": w.name, "batch": nb, "history_tokens": max_len,
                   "n_min": params.n_min, "n_max": params.n_max, "k_max": k,
                   "min_count": list(params.min_count),
                   "min_percent": list(params.min_percent), "graph_steps": G,
                   "graph_sizes": graph_sizes},
        "graph_us_per_step": round(gpu_us, 3),
        "mean_draft_tokens": round(float(ref[1].mean()), 3),
        "drafted_tokens_per_step": int(ref[1].sum()),
        "ns_per_drafted_token": round(gpu_us * 1e3 / max(1, int(ref[1].sum())), 3),
        "build": {"tokens": int(w.total_tokens), "ms": round(build_s * 1e3, 3),
                  "tokens_per_s": round(w.total_tokens / build_s, 1)},
    }
    if not args.no_cpu_baseline:
        import oracle
        op = oracle.NgramParams()
        n, t_start = 0, time.perf_counter()
        parity = True
        while n < G and time.perf_counter() - t_start < args.cpu_seconds:
            od, ol, ov = oracle.ngram_draft(op, w.histories, k)
            parity &= (np.array_equal(od, ref[0]) and np.array_equal(ol, ref[1])
                       and np.array_equal(ov, ref[2]))
            n += 1
        el = time.perf_counter() - t_start
        rec["cpu_baseline"] = {
            "value": round(n / el, 3), "unit": "draft steps/s", "cores": 1, "kind": "oracle",
            "sample": f"{n} repeats of the batch's drafts (brute-force recount, {el:.1f} s, "
                      f"one thread, {cpu_model()})"}
        rec["parity"] = "bit-exact" if parity else "MISMATCH"
        if not parity:
            print(json.dumps(rec))
            sys.exit(1)
    print(json.dumps(rec), flush=True)


def bench_stream(args, torch, B, wl, dev):
    """The streaming decode: 64 requests from 32,768 tokens, 1,024 steps of
    pld_draft_batch on the context's own store, then pld_append of the 1..16
    tokens each request accepted. The appended tokens follow each request's
    previous draft while it lasts, then fresh Zipf tokens.

    The oracle runs first, over all 1,024 steps (the CPU baseline leg): its
    drafts fix the append stream, and every GPU step is compared with it.
    With --no-cpu-baseline the GPU's own drafts fix the stream instead. One
    untimed eager pass on the GPU follows that stream; then all 1,024 steps
    are captured in a HIP graph and replayed from the same start state."""
    start_len = args.stream_start or wl.STREAM_START_LEN
    start = wl.config5_start(start_len)
    nb, steps_n, width = start.batch, wl.STREAM_STEPS, wl.STREAM_MAX_APPEND
    max_len = start_len + steps_n * width
    toks = np.zeros((steps_n, nb, width), np.int32)
    cnts = np.zeros((steps_n, nb), np.int32)

    # ---- the oracle's closed loop (CPU baseline leg) -------------------------
    want, cpu = None, None
    if not args.no_cpu_baseline:
        import oracle
        hs = [h.copy() for h in start.histories]
        op = oracle.NgramParams()
        want, cpu_s = [], 0.0
        for step in range(steps_n):
            t_ = time.perf_counter()
            if args.ngram:
                od, ol, om = oracle.ngram_draft(op, hs, start.k_max)
            else:
                od, ol, om, _ = oracle.draft(hs, start.n_min, start.n_max, start.k_max)
            cpu_s += time.perf_counter() - t_
            want.append((od, ol, om))
            counts, fresh = wl.stream_step_draws(step)
            toks[step] = wl.compose_append(od, ol, counts, fresh)
            cnts[step] = counts
            t_ = time.perf_counter()
            hs = oracle.append(hs, toks[step], cnts[step])
            cpu_s += time.perf_counter() - t_
        cpu = {"value": round(steps_n / cpu_s, 3), "unit": "draft steps/s", "cores": 1,
               "kind": "oracle",
               "sample": f"all {steps_n} streaming steps (draft + append, "
                         f"{'successor-count' if args.ngram else 'lookup'} oracle, "
                         f"{cpu_s:.1f} s, one thread, {cpu_model()})"}

    if args.index:
        ctx = B.pld_create_indexed(nb, max_len, start.n_min, start.n_max)
    elif args.ngram:
        ctx = B.pld_create_ngram(nb, max_len)
    else:
        ctx = B.pld_create(nb, max_len, own_store=True)
    rows, lens = B.pld_histories(ctx)
    if not (args.index or args.ngram):
        B.pld_configure(ctx, args.tile, args.fused)
    tile = None if (args.index or args.ngram) else B.pld_scan_tile(ctx, nb)
    # controller inputs: every outcome "0 accepted in time 1.0" is valid for
    # any previous choice, so the captured steps need no host round trip
    cparams = B.pld_control_params_default()
    c_state = torch.zeros((nb, B.PLD_CONTROL_STATE_WORDS), dtype=torch.float64, device=dev)
    c_acc = torch.zeros(nb, dtype=torch.int32, device=dev)
    c_time = torch.ones(nb, dtype=torch.float64, device=dev)
    c_src = torch.empty(nb, dtype=torch.int32, device=dev)

    def control():
        if args.control and not args.control_fused:
            B.pld_control(ctx, cparams, c_acc, c_time, out[1], out[2], c_state, nb, c_src)

    nparams = B.pld_ngram_params_default()

    def draft():
        if args.ngram:
            B.pld_draft_ngram(ctx, nparams, nb, start.k_max, out[0], out[1], levels)
        elif args.index:
            B.pld_draft_store(ctx, nb, start.n_min, start.n_max, start.k_max, out[0], out[1],
                              out[2])
        elif args.control_fused:
            B.pld_draft_control_batch(ctx, rows, lens, nb, start.n_min, start.n_max,
                                      start.k_max, out[0], out[1], out[2], cparams, c_acc,
                                      c_time, c_state, c_src)
        else:
            B.pld_draft_batch(ctx, rows, lens, nb, start.n_min, start.n_max, start.k_max,
                              out[0], out[1], out[2])
    init = torch.from_numpy(np.stack(start.histories)).to(dev)
    init_counts = torch.full((nb,), start_len, dtype=torch.int32, device=dev)
    out = B.alloc_outputs(nb, start.k_max, device=dev)
    levels = torch.zeros((nb, start.k_max), dtype=torch.int32, device=dev)

    def restart():
        B.pld_store_reset(ctx)
        B.pld_append(ctx, init, start_len, init_counts, nb)

    # ---- untimed eager pass: every step's drafts, on the fixed stream -------
    restart()
    lengths = np.full(nb, start_len, np.int64)
    total_tokens = 0
    mismatch, mean_len = None, []
    for step in range(steps_n):
        draft()
        d, l = out[0].cpu().numpy(), out[1].cpu().numpy()
        m = (levels if args.ngram else out[2]).cpu().numpy()
        mean_len.append(float(l.mean()))
        if want is None:
            counts, fresh = wl.stream_step_draws(step)
            toks[step] = wl.compose_append(d, l, counts, fresh)
            cnts[step] = counts
        elif mismatch is None and not (np.array_equal(d, want[step][0])
                                       and np.array_equal(l, want[step][1])
                                       and np.array_equal(m, want[step][2])):
            mismatch = step
        total_tokens += int(lengths.sum())
        lengths += cnts[step]
        B.pld_append(ctx, torch.from_numpy(toks[step]).to(dev), width,
                     torch.from_numpy(cnts[step]).to(dev), nb)
    assert B.pld_sync(ctx) == B.PLD_OK
    final_ref = [t.clone() for t in out[:3]]
    toks_d = torch.from_numpy(toks).to(dev)
    cnts_d = torch.from_numpy(cnts).to(dev)

    # one graph holds all 1,024 steps, in the eager pass's order: draft,
    # then append the tokens that step accepted
    cap = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    restart()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=cap):
        if args.append_draft:
            # draft(0), then append(s) + draft(s + 1) per call, then the last append
            draft()
            control()
            for step in range(steps_n - 1):
                if args.ngram:
                    B.pld_append_draft_ngram(ctx, toks_d[step], width, cnts_d[step], nb,
                                             nparams, start.k_max, out[0], out[1], levels)
                else:
                    B.pld_append_draft_store(ctx, toks_d[step], width, cnts_d[step], nb,
                                             start.n_min, start.n_max, start.k_max, out[0],
                                             out[1], out[2])
                control()
            B.pld_append(ctx, toks_d[steps_n - 1], width, cnts_d[steps_n - 1], nb)
        else:
            for step in range(steps_n):
                draft()
                control()
                B.pld_append(ctx, toks_d[step], width, cnts_d[step], nb)

    # whole replays of the 1,024-step graph: enough to cover the requested
    # warm-up and timed steps
    warm_reps = -(-args.warmup // steps_n)
    reps = max(1, -(-args.steps // steps_n))
    times = []
    for rep in range(warm_reps + reps):
        restart()
        torch.cuda.synchronize()
        e0 = torch.cuda.Event(enable_timing=True)
        e1 = torch.cuda.Event(enable_timing=True)
        t0 = time.perf_counter()
        e0.record()
        graph.replay()
        e1.record()
        torch.cuda.synchronize()
        wall = time.perf_counter() - t0
        for a_, b_ in zip(final_ref, out[:3]):
            assert torch.equal(a_, b_), "graph replay differs from the eager pass"
        if rep >= warm_reps:
            times.append((wall, e0.elapsed_time(e1) * 1e-3))
    assert B.pld_sync(ctx) == B.PLD_OK
    B.pld_destroy(ctx)
    if args.calibrate_copy:
        calibration_copies(torch, dev)
    wall = float(np.median([t[0] for t in times]))
    gpu_s = float(np.median([t[1] for t in times]))
    bytes_mean = 4.0 * total_tokens / steps_n
    rec = {
        "metric": METRIC,
        "value": round(steps_n / wall, 1),
        "unit": "draft steps/s",
        "n_gpus": 1,
        "steps": steps_n * len(times),
        "warmup": steps_n * warm_reps,
        "ms_per_step": round(wall * 1e3 / steps_n, 6),
        "higher_is_better": True,
        "scaling": "weak",
        "vs_baseline": None,
        "dtype": "int32",
        "data": "synthetic",
        "time_source": ("value, ms_per_step: host clock around one replay of the 1,024-step "
                        "graph (median over the timed replays), with a device synchronize on "
                        "each side; us_per_step_append_plus_draft and roofline: HIP events "
                        "on the launch stream around the same replays"),
        "config": {"workload": start.name, "batch": nb, "start_tokens": start_len,
                   "steps": steps_n, "n_min": start.n_min, "n_max": start.n_max,
                   "k_max": start.k_max, "mean_bytes_per_step": round(bytes_mean),
                   "drafting": ("successor-count cache" if args.ngram else
                                "n-gram index" if args.index else "scan"),
                   "calls_per_step": ((1 if args.append_draft else 2)
                                      + int(args.control and not args.control_fused)),
                   "controller": ("in the draft's launch" if args.control_fused else
                                  "own launch" if args.control else None),
                   "tile_tokens": tile,
                   "append_stream": ("the oracle's drafts" if want is not None
                                     else "the GPU's own drafts (no oracle run)")},
        "us_per_step_append_plus_draft": round(gpu_s * 1e6 / steps_n, 3),
        # for the index: the history bytes a scan would have read, per second
        ("scan_equivalent_GBps" if args.index else "scan_GBps"):
            round(bytes_mean * steps_n / gpu_s / 1e9, 1),
        "hbm_frac": None if (args.index or args.ngram) else
            round(bytes_mean * steps_n / gpu_s / 1e9 / HBM_PEAK_GBPS, 4),
    }
    if args.steps % steps_n or args.warmup % steps_n:
        rec["steps_requested"], rec["warmup_requested"] = args.steps, args.warmup
    if not (args.index or args.ngram):
        one_launch = args.append_draft and not (args.control and not args.control_fused)
        plain = (not args.control and start_len == wl.STREAM_START_LEN
                 and args.tile in (0, tile) and args.fused in (-1, 1))
        prof = (PROFILE_APPEND_DRAFT if one_launch else PROFILE_STREAM) if plain else None
        kernels = (["pld_scan"] + ([] if args.append_draft else ["pld_append_kernel"])
                   + (["pld_control_kernel"] if args.control and not args.control_fused else []))
        rec["roofline"] = {
            "bound": "hbm", "achieved": rec["scan_GBps"], "peak": HBM_PEAK_GBPS,
            "unit": "GB/s", "frac": rec["hbm_frac"],
            "traffic": profiled_traffic(prof),
            "traffic_by_request_size": profiled_traffic(prof, "traffic-sized-bytes-per-launch"),
            "traffic_note": TRAFFIC_NOTE + "; the median dispatch of the 1,024 steps, whose "
                            "history bytes grow step by step",
            "kernel": (" + ".join(kernels) + (" (the append in the scan's launch: one "
                                              "launch per step)" if one_launch else
                                              " (whole step)")),
            "time_source": f"HIP events around the replayed {steps_n}-step graph "
                           f"({len(kernels)} launch{'es' if len(kernels) > 1 else ''} a step"
                           f"{', plus the last append' if args.append_draft else ''}); "
                           "bytes = the mean history bytes per step"}
    if args.ngram:
        # a different drafter: no history bytes are read per step
        rec["metric"] = METRIC_NGRAM
        del rec["scan_GBps"]
        rec["config"]["n_min"], rec["config"]["n_max"] = nparams.n_min, nparams.n_max
        rec["mean_draft_tokens"] = round(float(np.mean(mean_len)), 3)
    if cpu is not None:
        rec["cpu_baseline"] = cpu
        rec["parity"] = ("bit-exact" if mismatch is None else "MISMATCH")
        rec["parity_steps"] = (f"all {steps_n} steps" if mismatch is None
                               else f"first mismatch at step {mismatch}")
        if mismatch is not None:
            print(json.dumps(rec))
            sys.exit(1)
    print(json.dumps(rec), flush=True)


# the verify step's geometry: one attention layer of a target model
STEP_HEADS, STEP_KV_HEADS, STEP_DIM, STEP_PAGE, STEP_VOCAB = 32, 8, 128, 64, 151936


def bench_verify_step(args, torch, B, wl, dev):
    """One verify step of 64 requests at workload 5's start lengths, on fixed
    histories: pld_draft_batch, then one layer's pld_kv_append and pld_attend
    over a paged bf16 cache of random keys and values, then pld_verify on
    random logits that hold the drafted tokens at a probability of about 0.8.
    The calls are captured into one graph and replayed; each is also timed in
    a graph of its own. Outputs of every replay equal the eager call's."""
    start = wl.config5_start(args.stream_start or wl.STREAM_START_LEN)
    nb, k, rows = start.batch, start.k_max, start.k_max + 1
    hq, hk, dim, page, vocab = STEP_HEADS, STEP_KV_HEADS, STEP_DIM, STEP_PAGE, STEP_VOCAB
    db = B.DeviceBatch(start.histories)
    ctx = B.pld_create(nb, db.max_len)
    p = B.pld_target_params_default()
    p.max_batch, p.max_rows, p.max_len = nb, rows, db.max_len + k
    p.q_heads, p.kv_heads, p.head_dim, p.page_tokens, p.vocab = hq, hk, dim, page, vocab
    p.rope.rot_dim = dim
    target = B.pld_create_target(p)
    gen = torch.Generator(device=dev)
    gen.manual_seed(11)
    bf16, i32 = torch.bfloat16, torch.int32
    width = -(-(db.max_len + k) // page)
    pages = nb * width
    table = torch.randperm(pages, generator=gen, device=dev).to(i32).view(nb, width)
    kc = torch.empty((pages, hk, page, dim), dtype=bf16, device=dev)
    vc = torch.empty((pages, hk, dim, page), dtype=bf16, device=dev)
    for cells in (kc, vc):
        for i in range(0, pages, 4096):
            cells[i:i + 4096].normal_(generator=gen)
    qkv = torch.randn((nb * rows, (hq + 2 * hk) * dim), generator=gen, device=dev).to(bf16)
    q = torch.empty((nb * rows, hq * dim), dtype=bf16, device=dev)
    attended = torch.zeros_like(q)
    draft, dlen, match, _ = B.alloc_outputs(nb, k, device=dev)
    uniform = torch.rand((nb, rows), generator=gen, device=dev)
    tokens = torch.empty((nb, rows), dtype=i32, device=dev)
    accepted, counts = (torch.empty(nb, dtype=i32, device=dev) for _ in range(2))
    logits = torch.empty((nb, rows, vocab), dtype=bf16, device=dev)

    def do_draft():
        B.pld_draft_batch(ctx, db.rows, db.lengths, nb, start.n_min, start.n_max, k, draft, dlen,
                          match)

    def do_append():
        w = qkv.shape[1]
        B.pld_kv_append(target, qkv, w, qkv[:, hq * dim:], qkv[:, (hq + hk) * dim:], w, rows,
                        db.lengths, dlen, nb, table, width, kc, vc, pages, None, None, q)

    def do_attend():
        B.pld_attend(target, q, hq * dim, rows, db.lengths, dlen, 0, nb, table, width, kc, vc,
                     pages, None, None, 0.0, 0, attended)

    def do_verify():
        B.pld_verify(target, logits, vocab, rows, draft, dlen, None, None, 0, None, uniform, nb,
                     tokens, accepted, counts)
    do_draft()
    for b in range(nb):
        z = torch.randn((rows, vocab), generator=gen, device=dev) * 2.0
        x = draft[b].clamp(min=0).long()[:, None]
        z[:k].scatter_(1, x, torch.logsumexp(z[:k], 1, keepdim=True) + 1.4)
        logits[b] = z.to(bf16)
    steps = {"draft": do_draft, "kv_append": do_append, "attend": do_attend, "verify": do_verify}

    def do_step():
        for f in steps.values():
            f()
    do_step()
    assert B.pld_sync(ctx) == B.PLD_OK and B.pld_sync(target) == B.PLD_OK
    want = [t.clone() for t in (attended, tokens, accepted)]

    def timed(f, reps):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
            f()
        for _ in range(max(1, args.warmup if reps == args.steps else 3)):
            graph.replay()
        torch.cuda.synchronize()
        e0, e1 = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        t0 = time.perf_counter()
        e0.record()
        for _ in range(reps):
            graph.replay()
        e1.record()
        torch.cuda.synchronize()
        wall = time.perf_counter() - t0
        for a_, b_ in zip(want, (attended, tokens, accepted)):
            assert torch.equal(a_, b_), "graph replay differs from the eager pass"
        return wall, e0.elapsed_time(e1) * 1e-3
    wall, gpu_s = timed(do_step, args.steps)
    part = {name: timed(f, min(200, args.steps))[1] / min(200, args.steps) * 1e6
            for name, f in steps.items()}
    assert B.pld_sync(ctx) == B.PLD_OK and B.pld_sync(target) == B.PLD_OK
    seen = int((db.lengths + dlen).sum())
    cache_bytes = seen * hk * dim * 2 * 2
    rec = {
        "metric": "verify steps/s; us per call of the step",
        "value": round(args.steps / wall, 1), "unit": "verify steps/s", "n_gpus": 1,
        "steps": args.steps, "warmup": args.warmup,
        "ms_per_step": round(wall * 1e3 / args.steps, 6), "higher_is_better": True,
        "scaling": "weak", "vs_baseline": None, "dtype": "bf16", "data": "synthetic",
        "config": {"workload": start.name, "batch": nb, "q_heads": hq, "kv_heads": hk,
                   "head_dim": dim, "page_tokens": page, "vocab": vocab, "rows": rows,
                   "layers": 1, "mean_draft": round(float(dlen.float().mean()), 2),
                   "mean_accepted": round(float(accepted.float().mean()), 2)},
        "us_per_step": round(gpu_s * 1e6 / args.steps, 2),
        "us_per_call": {n: round(t, 2) for n, t in part.items()},
        "attend_cache_GBps": round(cache_bytes / part["attend"] / 1e3, 1),
        "time_source": "value, ms_per_step: host clock around the replays, a device synchronize "
                       "on each side; us_*: HIP events on the launch stream",
    }
    B.pld_destroy(ctx)
    B.pld_destroy(target)
    print(json.dumps(rec), flush=True)


if __name__ == "__main__":
    main()
