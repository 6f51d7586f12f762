"""Benchmark: microseconds per MoE dispatch+combine on one MI355X, and the
achieved HBM bandwidth against the 8 TB/s peak.

One step = moe_dispatch_send + moe_dispatch_recv + moe_combine_send +
moe_combine_recv over one batch of the DeepSeek-R1-shaped decode workload
(32 logical ranks x 128 tokens, hidden 7168 bf16, top-8 of 256 experts).  The
expert between dispatch and combine is outside the path: its output (the
stand-in y = x*(e+1) of the first cycle) is computed once before timing and
reused, since the routing is the same every step.  Inputs are resident in HBM
before the timed region.

Timing protocol: `warmup` untimed steps; then `steps` steps back to back
under a wall clock (the warm figure, reported beside the headline); then the
timed region, `steps` steps each started with the MALL flushed (a 512 MB
buffer written first) and bracketed by events: `value` is the median of those
per-step times (µs), with p10 / p90 beside it.

Prints one JSON line.  Kernel durations come from HIP events the library
attaches to the kernel dispatches: every kernel in an untimed pass (the
`kernels` table, which picks the dominant kernel), then only the dominant
kernel during the timed steps (its `roofline` entry), since each timed kernel
adds a few microseconds of gap to the step.  The CPU baseline is the oracle
on the same workload, single-threaded and split over the host's cores.
"""
from __future__ import annotations

import argparse
import ctypes
import hashlib
import json
import os
import sys
import time

ROOT = os.path.dirname(os.path.abspath(__file__))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

METRIC = "µs per dispatch+combine and achieved HBM GB/s (% of peak), DeepSeek-R1 shape"
HBM_PEAK_GBPS = 8000.0


def partial_rows(cfg, idx) -> int:
    """P: the number of distinct (token, destination rank) pairs, i.e. the rows
    the expert-side partial combine returns."""
    import numpy as np
    N, T = cfg.N, cfg.T
    d = np.asarray(idx, dtype=np.int64) // cfg.L                    # [N][T][K]
    tok = np.arange(N * T, dtype=np.int64).reshape(N, T, 1)
    return int(np.unique(tok * N + d).size)


# A sender's tokens up to this size make the pack run in send-row order (the
# library's rule).
PACK_ROWS_MAX_SENDER_BYTES = 2 << 20
# With the partial combine and the send-row-order pack, the pack's record
# blocks form their sender's bases from sums over the senders up to this many
# terms per block, (E + 2N + 2) * N (the library's rule); past it the route
# plan forms the group tables.
RECORD_SUMS_MAX = 1 << 16


def plan_forms_offsets(cfg, combine: str = "receiver", layout: str = "packed") -> bool:
    """Whether the route plan's last workgroup forms the group offsets (the
    library's rule): for the token-order pack unless its rows go to fixed
    slots with the receiver-side combine, and for the partial combine's
    records in the send-row-order pack past RECORD_SUMS_MAX."""
    partial = combine == "partial"
    if cfg.T * cfg.H * 2 > PACK_ROWS_MAX_SENDER_BYTES:
        return partial or layout != "fixed"
    return partial and (cfg.E + 2 * cfg.N + 2) * cfg.N > RECORD_SUMS_MAX


def kernel_bytes(cfg, transport: str = "staged", combine: str = "receiver", P: int = 0,
                 layout: str = "packed") -> dict:
    """Algorithmic HBM bytes per launch of each kernel: every buffer the method
    mandates is written once and read once by the next stage; inputs are read
    once per token.  The int32 row maps the pack kernel writes for the later
    movers (4-8 bytes per row of 7-14 KiB) are an implementation detail and not
    counted.  With the partial combine (P partial rows), the router weights
    travel with the dispatched rows and combine moves P rows instead of R.
    The receiver's map kernel forms the group offsets from the exchanged
    counts and send offsets and writes its maps, 20 bytes per row (24 with
    fixed slots): tables and maps are its whole job, so they are counted
    there.  The route plan's last workgroup forms the group offsets too (the
    same tables in and out) only where a kernel before dispatch_recv needs
    them (plan_forms_offsets; the map kernel then reads them instead,
    counted alike).
    When the pack runs in send-row order (a sender's tokens within 2 MiB) the
    route plan writes each send row's item and the pack reads it in place of
    the positions (staged: the send meta words, which the pack no longer
    writes; direct: the pack no longer reads idx)."""
    N, T, K, E, H = cfg.N, cfg.T, cfg.K, cfg.E, cfg.H
    R = N * T * K
    fp8 = cfg.dtype == "fp8"
    hb = H if fp8 else 2 * H                     # payload bytes per row
    sb = (H // 128) * 4 if fp8 else 0            # block scales per row
    hy = 2 * H                                   # combine row
    tokens = N * T
    row_order = T * H * 2 <= PACK_ROWS_MAX_SENDER_BYTES
    # the group offsets: counts and send offsets in; receive offsets, receive
    # bases and expert offsets out
    offs = (N * E * 4 + N * (E + 1) * 4 + N * (N + 1) * 4 + (N + 1) * 4 + (E + 1) * 4)
    kb = {
        # idx in; counts, send offsets (both orientations), positions out
        "route_plan": R * 4 + N * E * 4 + 2 * N * (E + 1) * 4 + R * 4,
        "pack": tokens * H * 2 + R * 4 * 2 + R * (hb + sb + 4),
        "transfer": 2 * R * (hb + sb + 4),
        "shuffle": R * (hb + sb + 4) + R * (hb + sb + 8) + (E + 1) * 4,
        "combine_pack": 2 * R * hy,
        "transfer_back": 2 * R * hy,
        "combine_reduce": R * hy + R * 8 + tokens * H * 2,
        "recv_map": offs + R * (20 + (4 if layout == "fixed" else 0)),
    }
    tail = plan_forms_offsets(cfg, combine, layout)
    if tail:
        kb["route_plan"] += offs
    if row_order:
        kb["route_plan"] += R * 4
        kb["pack"] -= R * 4
    if transport == "direct":
        # pack writes the receive rows itself and combine writes the return
        # rows itself: no transfer passes
        for k in ("transfer", "combine_pack", "transfer_back"):
            del kb[k]
        kb["combine_push"] = 2 * R * hy
    if combine == "partial":
        # second route-plan pass: rank and position of every item and the
        # partial rows' send offsets (both orientations); where it forms the
        # group tables, also the partial rows' owner offsets and bases and
        # each sender's base row (E + 2N + 2 ints: its first expert rows,
        # first receive and owner-layout partial rows on each rank, first
        # token-layout partial row, P), else the map kernel forms the bases
        # (owner and token layout) from the send offsets; weights (4 bytes a
        # row) through pack and transfer
        kb["route_plan"] += 2 * R * 4 + 2 * N * (N + 1) * 4
        if tail:
            kb["route_plan"] += N * (E + 2 * N + 2) * 4 + 2 * N * (N + 1) * 4 + 2 * (N + 1) * 4
        else:
            kb["recv_map"] += N * (N + 1) * 4 + 2 * (N + 1) * 4
        kb["pack"] += 2 * R * 4
        if "transfer" in kb:
            kb["transfer"] += 2 * R * 4
        for k in ("combine_pack", "transfer_back", "combine_push", "combine_reduce"):
            kb.pop(k, None)
        # expert rows in (+ per item its weight; per partial row its 32-byte
        # record, which names the rows of its first two items: the item-table
        # reads of larger partials are not counted, like the row maps),
        # partial rows out
        kb["partial_send"] = R * hy + R * 4 + P * 32 + P * hy
        if transport == "staged":
            kb["partial_transfer"] = 2 * P * hy
        kb["partial_reduce"] = P * hy + R * 8 + tokens * H * 2
    return kb


def _code_only(text: str) -> str:
    """C/C++ source with comments removed and whitespace collapsed, so that
    editing a comment does not count as changing a kernel."""
    out, i, n = [], 0, len(text)
    while i < n:
        if text.startswith("//", i):
            j = text.find("\n", i)
            i = n if j < 0 else j
        elif text.startswith("/*", i):
            j = text.find("*/", i + 2)
            i = n if j < 0 else j + 2
            out.append(" ")
        elif text[i] == '"':
            j = i + 1
            while j < n and text[j] != '"':
                j += 2 if text[j] == "\\" else 1
            out.append(text[i:j + 1])
            i = j + 1
        else:
            out.append(text[i])
            i += 1
    return " ".join("".join(out).split())


# the sources of the dispatch/combine path, whose traffic the profiles record
PATH_SOURCES = ("moe_ep.hip", "moe_kernels.h", "moe_kernels.hip")


def kernel_source_hash() -> str:
    """Hash of the path's sources, comments and whitespace ignored."""
    h = hashlib.sha256()
    csrc = os.path.join(ROOT, "combine_moe_dispatch_amd", "csrc")
    for name in PATH_SOURCES:
        with open(os.path.join(csrc, name), encoding="utf-8") as f:
            h.update(name.encode() + _code_only(f.read()).encode())
    return h.hexdigest()[:16]


def traffic_key(args) -> str:
    """Name of the counter summary of a workload and mode: the workload key,
    then _direct, _partial and _fixed for the non-default choices (each mode
    moves different rows, so each has its own summary)."""
    return (args.config + ("" if args.transport == "staged" else "_direct")
            + ("_partial" if args.combine == "partial" else "")
            + ("_fixed" if getattr(args, "layout", "packed") == "fixed" else ""))


def measured_traffic(config_key: str, kernel: str, src_hash: str):
    """HBM bytes per launch from the committed rocprofv3 counter summary, if it
    was taken on the current kernel sources; else None."""
    path = os.path.join(ROOT, "profiles", f"traffic_{config_key}.json")
    try:
        with open(path) as f:
            rec = json.load(f)
    except (OSError, ValueError):
        return None
    if rec.get("source_hash") != src_hash:
        return None
    k = rec.get("kernels", {}).get(kernel)
    return None if k is None else k.get("hbm_bytes_per_launch")


# ---------------------------------------------------------------- profiles

CAL_BYTES = 469_762_048        # one plain device copy of this many bytes each way
KERNEL_OF = [("route_plan_kernel", "route_plan"), ("pack_bf16_kernel", "pack"),
             ("combine_push_kernel", "combine_push"),
             ("pack_fp8_kernel", "pack"), ("transfer_back_kernel", "transfer_back"),
             ("transfer_kernel", "transfer"), ("shuffle_kernel", "shuffle"),
             ("combine_pack_kernel", "combine_pack"),
             ("combine_reduce_kernel", "combine_reduce"),
             ("partial_send_kernel", "partial_send"),
             ("partial_transfer_kernel", "partial_transfer"),
             ("partial_reduce_kernel", "partial_reduce"),
             ("recv_map_kernel", "recv_map"), ("pack_rows_bf16_kernel", "pack"),
             ("pack_rows_fp8_kernel", "pack"), ("pack_rows_rec_bf16_kernel", "pack"),
             ("pack_rows_rec_fp8_kernel", "pack")]


def _kernel_key(name: str):
    for sym, key in KERNEL_OF:
        if f"::{sym}<" in name or f"::{sym}(" in name:
            return key
    return None


def copy_calibration() -> int:
    """A plain device copy of CAL_BYTES bytes, 5 times (torch's copy kernel):
    the reference for scaling rocprofv3's FETCH_SIZE / WRITE_SIZE counters."""
    import torch
    src = torch.empty(CAL_BYTES, dtype=torch.uint8, device="cuda")
    src.fill_(7)
    dst = torch.empty_like(src)
    for _ in range(5):
        dst.copy_(src)
    torch.cuda.synchronize()
    print(json.dumps({"calibration_copy_bytes": CAL_BYTES, "launches": 5}), flush=True)
    return 0


def _counter_by_kernel(db: str, counter: str) -> dict:
    import sqlite3
    con = sqlite3.connect(db)
    rows = con.execute("select kernel_name, value from counters_collection where counter_name=?",
                       (counter,)).fetchall()
    acc = {}
    for name, v in rows:
        acc.setdefault(name, []).append(float(v))
    return acc


def traffic_from(cfg, fetch_db, write_db, cal_fetch_db, cal_write_db, transport="staged",
                 combine="receiver") -> dict:
    """HBM bytes per launch of each kernel from two rocprofv3 --pmc runs
    (FETCH_SIZE, WRITE_SIZE; KiB per dispatch), each scaled by what the same
    counter reads for the plain copy of CAL_BYTES bytes."""
    def cal_factor(db, counter):
        acc = _counter_by_kernel(db, counter)
        # the calibration copy: the kernel with >= 5 dispatches and the largest reading
        name = max((k for k, v in acc.items() if len(v) >= 5), key=lambda k: sum(acc[k]))
        kib = sum(acc[name]) / len(acc[name])
        return CAL_BYTES / (kib * 1024.0)
    ff = cal_factor(cal_fetch_db, "FETCH_SIZE")
    wf = cal_factor(cal_write_db, "WRITE_SIZE")
    kb = kernel_bytes(cfg, transport, combine, _partial_rows_of(cfg, combine))
    out = {}
    for counter, db, f, field in (("FETCH_SIZE", fetch_db, ff, "fetch_bytes"),
                                  ("WRITE_SIZE", write_db, wf, "write_bytes")):
        for name, vals in _counter_by_kernel(db, counter).items():
            key = _kernel_key(name)
            if key is None:
                continue
            rec = out.setdefault(key, {"launches": len(vals)})
            rec[field] = round(sum(vals) / len(vals) * 1024.0 * f)
    for key, rec in out.items():
        rec["hbm_bytes_per_launch"] = rec.get("fetch_bytes", 0) + rec.get("write_bytes", 0)
        rec["algorithmic_bytes_per_launch"] = kb[key]
        rec["ratio"] = round(rec["hbm_bytes_per_launch"] / kb[key], 4)
    return {"workload": cfg.describe(), "source_hash": kernel_source_hash(),
            "fetch_factor": round(ff, 4), "write_factor": round(wf, 4), "kernels": out}


def _partial_rows_of(cfg, combine: str) -> int:
    if combine != "partial":
        return 0
    from workloads import make_routing
    return partial_rows(cfg, make_routing(cfg)[0])


def trace_summary(cfg, db: str, timed=None, layout: str = "packed") -> str:
    """Markdown table of the library's kernels from a rocprofv3 kernel trace.
    With timed = (steps, warmup) of the traced bench command, a column with
    each kernel's average over the launches of its timed region (the
    MALL-flushed steps): per kernel, launch 1 is the first cycle, then warmup
    steps, max(10, warmup) all-kernel timing steps, `steps` warm steps, then
    the `steps` timed ones."""
    import sqlite3
    con = sqlite3.connect(db)
    acc = {}
    for name, dur in con.execute("select name, duration from kernels order by start"):
        key = _kernel_key(name)
        if key is not None:
            acc.setdefault(key, []).append(dur / 1000.0)
    first = None if timed is None else 1 + timed[1] + max(10, timed[1]) + timed[0]
    head = "| kernel | launches | avg us | min us | max us | algorithmic GB/s |"
    rule = "|---|---|---|---|---|---|"
    if first is not None:
        head += " timed-region avg us |"
        rule += "---|"
    lines = [head, rule]
    transport = "staged" if "transfer" in acc else "direct"
    combine = "partial" if "partial_send" in acc else "receiver"
    kb = kernel_bytes(cfg, transport, combine, _partial_rows_of(cfg, combine), layout)
    for key in ["route_plan", "pack", "transfer", "recv_map", "shuffle",
                "combine_pack", "transfer_back", "combine_push", "combine_reduce",
                "partial_send", "partial_transfer", "partial_reduce"]:
        if key in acc:
            v = acc[key]
            avg = sum(v) / len(v)
            line = (f"| {key} | {len(v)} | {avg:.2f} | {min(v):.2f} | {max(v):.2f} | "
                    f"{kb[key] / (avg * 1e-6) / 1e9:.0f} |")
            if first is not None:
                t = v[first:first + timed[0]]
                line += f" {sum(t) / len(t):.2f} |" if t else " - |"
            lines.append(line)
    return "\n".join(lines)


def traffic_xcheck(cfg, dram_db, cal_dram_db, req_db, cal_req_db, traffic_json) -> dict:
    """HBM bytes per launch from two more counter families, each calibrated on
    the plain copy of CAL_BYTES each way, beside the FETCH_SIZE/WRITE_SIZE
    figures of traffic_json: (a) requests to DRAM (TCC_EA0_RDREQ_DRAM_sum,
    TCC_EA0_WRREQ_DRAM_sum) times the bytes per request the copy shows, (b)
    the raw EA requests (TCC_EA0_RDREQ_sum / _32B_sum, TCC_EA0_WRREQ_sum /
    _64B_sum) sized 32/64 bytes as FETCH_SIZE's formula does, scaled like it."""
    def per_kernel(db, ctr):
        acc = _counter_by_kernel(db, ctr)
        out = {}
        for name, vals in acc.items():
            k = _kernel_key(name)
            if k:
                out[k] = sum(vals) / len(vals)
        cal = max((v for v in acc.values() if len(v) >= 5), key=sum, default=None)
        return out, (sum(cal) / len(cal) if cal else None)
    rd = per_kernel(dram_db, "TCC_EA0_RDREQ_DRAM_sum")[0]
    wr = per_kernel(dram_db, "TCC_EA0_WRREQ_DRAM_sum")[0]
    b_rd = CAL_BYTES / per_kernel(cal_dram_db, "TCC_EA0_RDREQ_DRAM_sum")[1]
    b_wr = CAL_BYTES / per_kernel(cal_dram_db, "TCC_EA0_WRREQ_DRAM_sum")[1]
    names = ("TCC_EA0_RDREQ_sum", "TCC_EA0_RDREQ_32B_sum", "TCC_EA0_WRREQ_sum",
             "TCC_EA0_WRREQ_64B_sum")
    q = {c: per_kernel(req_db, c)[0] for c in names}
    cq = {c: per_kernel(cal_req_db, c)[1] for c in names}

    def rbytes(r, r32):
        return 32 * r32 + 64 * (r - r32)

    def wbytes(w, w64):
        return 64 * w64 + 32 * (w - w64)
    f_rd = CAL_BYTES / rbytes(cq[names[0]], cq[names[1]])
    f_wr = CAL_BYTES / wbytes(cq[names[2]], cq[names[3]])
    with open(traffic_json) as f:
        tj = json.load(f)
    rows = {}
    for k, rec in tj["kernels"].items():
        if k not in rd:
            continue
        dram = rd[k] * b_rd + wr[k] * b_wr
        ea = (rbytes(q[names[0]][k], q[names[1]][k]) * f_rd
              + wbytes(q[names[2]][k], q[names[3]][k]) * f_wr)
        fw = rec["hbm_bytes_per_launch"]
        rows[k] = {"fetch_write_size": fw, "dram_requests": round(dram), "ea_requests": round(ea),
                   "dram_over_fetch_write": round(dram / fw, 4),
                   "ea_over_fetch_write": round(ea / fw, 4)}
    return {"workload": cfg.describe(), "source_hash": kernel_source_hash(),
            "bytes_per_dram_read_request": round(b_rd, 3),
            "bytes_per_dram_write_request": round(b_wr, 3),
            "ea_read_factor": round(f_rd, 4), "ea_write_factor": round(f_wr, 4), "kernels": rows}


def _hip_runtime():
    """The HIP runtime already loaded by torch (found by soname, not loaded again)."""
    import torch  # noqa: F401  (loads the runtime)
    mode = getattr(os, "RTLD_NOLOAD", 4) | os.RTLD_LAZY
    for name in ("libamdhip64.so.7", "libamdhip64.so"):
        try:
            lib = ctypes.CDLL(name, mode=mode)
            break
        except OSError:
            lib = None
    assert lib is not None, "HIP runtime not loaded"
    lib.hipExtStreamCreateWithCUMask.argtypes = [ctypes.POINTER(ctypes.c_void_p), ctypes.c_uint32,
                                                 ctypes.POINTER(ctypes.c_uint32)]
    lib.hipExtStreamCreateWithCUMask.restype = ctypes.c_int
    lib.hipStreamDestroy.argtypes = [ctypes.c_void_p]
    lib.hipStreamDestroy.restype = ctypes.c_int
    return lib


def overlap_demo(cfg, args) -> dict:
    """Send/recv split in use: a bf16 GEMM standing in for the shared expert
    ([N*T, H] x [H, 2048]) runs on its own stream while dispatch-send runs;
    compared with running the two back to back on one stream."""
    import numpy as np
    import torch

    import combine_moe_dispatch_amd as mep
    from workloads import make_inputs
    inp = make_inputs(cfg)
    N, T, K, E, H = cfg.N, cfg.T, cfg.K, cfg.E, cfg.H
    R = cfg.rows
    transport = mep.MOE_TRANSPORT_DIRECT if args.transport == "direct" else mep.MOE_TRANSPORT_STAGED
    x = torch.from_numpy(inp["x"].view(np.int16)).cuda()
    idx = torch.from_numpy(inp["idx"]).cuda()
    expert_x = torch.empty((R, 2 * H), dtype=torch.uint8, device="cuda")
    offs = torch.empty((E + 1,), dtype=torch.int32, device="cuda")
    a = torch.randn((N * T, H), dtype=torch.bfloat16, device="cuda")
    b = torch.randn((H, 2048), dtype=torch.bfloat16, device="cuda")
    g = mep.moe_group_create(N, E, K, H, T, mep.MOE_BF16, transport)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    # a dispatch cycle must be completed before the next send; the combine
    # halves are run (untimed) with a fixed expert output
    y = torch.zeros((R, H), dtype=torch.bfloat16, device="cuda")
    w = torch.from_numpy(inp["w"]).cuda()
    out = torch.empty((N, T, H), dtype=torch.bfloat16, device="cuda")

    def finish(stream):
        mep.moe_combine_send(g, y, stream=stream)
        mep.moe_combine_recv(g, w, out, stream=stream)

    def timed(fn, iters):
        ts = []
        for _ in range(iters):
            torch.cuda.synchronize()
            t0 = time.perf_counter()
            fn()
            torch.cuda.synchronize()
            ts.append(time.perf_counter() - t0)
            finish(s1)
        torch.cuda.synchronize()
        return float(np.median(ts)) * 1e6

    def gemm_only():
        with torch.cuda.stream(s2):
            torch.matmul(a, b)

    def dispatch_only():
        mep.moe_dispatch_send(g, T, x, idx, stream=s1)
        mep.moe_dispatch_recv(g, expert_x, None, offs, stream=s1)

    def serial():
        mep.moe_dispatch_send(g, T, x, idx, stream=s1)
        with torch.cuda.stream(s1):
            torch.matmul(a, b)
        mep.moe_dispatch_recv(g, expert_x, None, offs, stream=s1)

    def overlapped():
        ev = torch.cuda.Event()
        with torch.cuda.stream(s2):
            torch.matmul(a, b)
            ev.record(s2)
        mep.moe_dispatch_send(g, T, x, idx, stream=s1)
        mep.moe_dispatch_recv(g, expert_x, None, offs, stream=s1)
        s1.wait_event(ev)

    # CU-partitioned streams: the movers on one set of CUs, the GEMM on the
    # rest (hipExtStreamCreateWithCUMask), so neither starves the other of
    # wave slots
    hip = _hip_runtime()
    ncu = torch.cuda.get_device_properties(0).multi_processor_count

    def cu_stream(first, count):
        words = (ncu + 31) // 32
        mask = (ctypes.c_uint32 * words)()
        for c in range(first, first + count):
            mask[c // 32] |= 1 << (c % 32)
        handle = ctypes.c_void_p()
        rc = hip.hipExtStreamCreateWithCUMask(ctypes.byref(handle), words, mask)
        assert rc == 0, rc
        return torch.cuda.ExternalStream(handle.value), handle

    def overlapped_partitioned(split):
        sa, ha = cu_stream(0, split)
        sb, hb = cu_stream(split, ncu - split)

        def run():
            ev = torch.cuda.Event()
            with torch.cuda.stream(sb):
                torch.matmul(a, b)
                ev.record(sb)
            mep.moe_dispatch_send(g, T, x, idx, stream=sa)
            mep.moe_dispatch_recv(g, expert_x, None, offs, stream=sa)
            sa.wait_event(ev)
        timed(run, 3)
        t = timed(run, 30)
        torch.cuda.synchronize()
        hip.hipStreamDestroy(ha)
        hip.hipStreamDestroy(hb)
        return t

    for fn in (dispatch_only, serial, overlapped):      # warm up
        timed(fn, 3)
    res = {"dispatch_us": timed(dispatch_only, 30), "serial_us": timed(serial, 30),
           "overlapped_us": timed(overlapped, 30)}
    torch.cuda.synchronize()
    ts = []
    for _ in range(30):
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        gemm_only()
        torch.cuda.synchronize()
        ts.append(time.perf_counter() - t0)
    res["gemm_us"] = float(np.median(ts)) * 1e6
    for split in (ncu // 2, 3 * ncu // 4):
        res[f"overlapped_cu_split_{split}_{ncu - split}_us"] = overlapped_partitioned(split)
    mep.moe_group_destroy(g)
    res = {k: round(v, 1) for k, v in res.items()}
    best = min(v for k, v in res.items() if k.startswith("overlapped"))
    res["hidden_fraction_of_gemm"] = round((res["serial_us"] - best) / res["gemm_us"], 3)
    res["workload"] = cfg.describe() + f" transport={args.transport}"
    res["other_work"] = f"bf16 GEMM [{N * T} x {H}] x [{H} x 2048] on its own stream"
    return res


def layer_run(cfg, args) -> dict:
    """A whole expert layer on the workload's tokens, with real experts of
    width args.expert_width: add + RMS norm, routing, e4m3 dispatch, gate/up
    and down products, combine.  Median time of every operator and of the
    layer, and of the few-token layer for a handful of the same tokens."""
    import numpy as np
    import torch

    import combine_moe_dispatch_amd as mep
    N, T, K, E, H, F = cfg.N, cfg.T, cfg.K, cfg.E, cfg.H, args.expert_width
    tokens, R = N * T, cfg.rows
    dev = torch.device("cuda", 0)
    gen = torch.Generator(device=dev)
    gen.manual_seed(cfg.seed)

    def empty(*shape, dt=torch.float32):
        return torch.empty(shape, dtype=dt, device=dev)

    def weights(n, k):
        w = empty(E, n, k, dt=torch.float8_e4m3fn)
        for e in range(E):
            w[e] = (96.0 * torch.randn((n, k), generator=gen, device=dev)).clamp_(-448, 448).to(w.dtype)
        return w, torch.full((E, n // 128, k // 128), 1.0 / (96.0 * k ** 0.5), device=dev)

    bf16, e4m3, i32 = torch.bfloat16, torch.float8_e4m3fn, torch.int32
    x = torch.randn((tokens, H), generator=gen, device=dev).to(bf16)
    res = torch.randn((tokens, H), generator=gen, device=dev).to(bf16)
    norm_w = torch.ones(H, dtype=bf16, device=dev)
    logits = torch.randn((tokens, E), generator=gen, device=dev)
    (w13, s13), (w2, s2) = weights(2 * F, H), weights(H, F)
    res_out, y, out = empty(tokens, H, dt=bf16), empty(tokens, H, dt=bf16), empty(tokens, H, dt=bf16)
    idx, w = empty(tokens, K, dt=i32), empty(tokens, K)
    ex, es, off = empty(R, H, dt=e4m3), empty(R, H // 128), empty(E + 1, dt=i32)
    h, hs, ey = empty(R, F, dt=e4m3), empty(R, F // 128), empty(R, H, dt=bf16)
    g = mep.moe_group_create(N, E, K, H, T, mep.MOE_FP8_E4M3)
    calls = {
        "add_rmsnorm": lambda: mep.moe_add_rmsnorm(tokens, H, x, res, norm_w, 1e-6, res_out, y, None, None),
        "topk_route": lambda: mep.moe_topk_route(tokens, E, K, logits, mep.MOE_FP32, True, idx, w),
        "dispatch": lambda: (mep.moe_dispatch_send(g, T, y, idx), mep.moe_dispatch_recv(g, ex, es, off)),
        "expert_gate_up": lambda: mep.moe_expert_gate_up(R, E, F, H, ex, es, off, w13, s13, h, hs),
        "expert_matmul": lambda: mep.moe_expert_matmul(R, E, H, F, h, hs, off, w2, s2, ey),
        "combine": lambda: (mep.moe_combine_send(g, ey), mep.moe_combine_recv(g, w, out)),
    }
    steps = min(args.steps, 50)
    marks = [[torch.cuda.Event(enable_timing=True) for _ in range(len(calls) + 1)] for _ in range(steps)]
    for n in range(args.warmup + steps):
        ev = marks[max(n - args.warmup, 0)]
        ev[0].record()
        for i, call in enumerate(calls.values()):
            call()
            ev[i + 1].record()
    torch.cuda.synchronize()
    if mep.moe_group_status(g) != mep.MOE_OK:
        raise RuntimeError("the layer's cycle failed")
    mep.moe_group_destroy(g)

    def median(pairs):
        return round(float(np.median([a.elapsed_time(b) for a, b in pairs])) * 1e3, 1)

    rec = {"metric": "expert layer", "unit": "us", "value": median([(m[0], m[-1]) for m in marks]),
           "us": {name: median([(m[i], m[i + 1]) for m in marks]) for i, name in enumerate(calls)},
           "few_token_us": {}, "workload": cfg.describe() + f" expert width {F}"}
    for n in (1, 8, 32):
        if n > min(tokens, mep.MOE_FEW_TOKENS_MAX):
            break
        ws = empty(mep.moe_few_token_workspace(n, K, H, F), dt=torch.uint8)
        ev = [torch.cuda.Event(enable_timing=True) for _ in range(steps + 1)]
        for i in range(args.warmup + steps + 1):
            if i >= args.warmup:
                ev[i - args.warmup].record()
            mep.moe_few_token_layer(n, E, K, H, F, y, idx, w, w13, s13, w2, s2, out, ws)
        torch.cuda.synchronize()
        rec["few_token_us"][str(n)] = median(list(zip(ev, ev[1:])))
    return rec


def hbm_ceiling(torch, mep, nbytes: int = 1 << 30, iters: int = 10, batches: int = 5) -> dict:
    """What HBM delivers to the library's streaming probes (16-byte
    nontemporal vectors, the movers' access style) on buffers of nbytes: a
    copy, a pure read and a pure write.  The rate depends on the footprint
    against the 256 MB MALL, so it is measured at the dominant kernel's own
    footprint and at 1 GiB.  Each rate is the best of `batches` timed batches
    of `iters` back-to-back launches (a single short batch varied by up to
    15% between runs)."""
    nbytes -= nbytes % 16
    src = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    src.fill_(1)
    dst = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    res = {}
    for name, kind, moved in (("copy", mep.MOE_PROBE_COPY, 2), ("read", mep.MOE_PROBE_READ, 1),
                              ("write", mep.MOE_PROBE_WRITE, 1)):
        for _ in range(2):
            mep.moe_hbm_probe(kind, dst, src, nbytes)
        torch.cuda.synchronize()
        best = None
        for _ in range(batches):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            for _ in range(iters):
                mep.moe_hbm_probe(kind, dst, src, nbytes)
            b.record()
            b.synchronize()
            ms = a.elapsed_time(b) / iters
            best = ms if best is None else min(best, ms)
        res[f"{name}_gbps"] = round(nbytes * moved / (best * 1e-3) / 1e9, 1)
    res["bytes"] = nbytes
    del src, dst
    return res


def step_distribution(torch, step, stream, n: int, flush_bytes: int = 0) -> dict:
    """Per-step times from an event pair around each step (p10 / p50 / p90, µs);
    with flush_bytes, a scratch buffer that size is written before every step
    so the step starts with the MALL holding none of its data."""
    scratch = torch.empty(flush_bytes, dtype=torch.uint8, device="cuda") if flush_bytes else None
    evs = [(torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True))
           for _ in range(n)]
    torch.cuda.synchronize()
    for a, b in evs:
        if scratch is not None:
            with torch.cuda.stream(stream):
                scratch.fill_(0)
        a.record(stream)
        step()
        b.record(stream)
    torch.cuda.synchronize()
    ts = sorted(a.elapsed_time(b) * 1e3 for a, b in evs)

    def q(p):
        return round(ts[min(len(ts) - 1, int(p * len(ts)))], 1)
    return {"p10": q(0.1), "p50": q(0.5), "p90": q(0.9), "n": n}


def host_cpu() -> dict:
    """The host's CPU as lscpu and the scheduler report it."""
    import subprocess
    info = {"logical_cpus": os.cpu_count(), "cpus_in_affinity": len(os.sched_getaffinity(0))}
    try:
        out = subprocess.run(["lscpu"], capture_output=True, text=True, timeout=10).stdout
        for line in out.splitlines():
            k, _, v = line.partition(":")
            k, v = k.strip(), v.strip()
            if k in ("Model name", "Vendor ID", "CPU family", "Model", "Socket(s)",
                     "Core(s) per socket", "Thread(s) per core", "CPU max MHz", "L3 cache"):
                info[k.lower().replace("(s)", "s").replace(" ", "_")] = v
    except (OSError, subprocess.SubprocessError):
        pass
    if "model_name" not in info:
        try:
            with open("/proc/cpuinfo") as f:
                for line in f:
                    if line.startswith("model name"):
                        info["model_name"] = line.split(":", 1)[1].strip()
                        break
        except OSError:
            pass
    return info


# host threads for the oracle's threaded leg: the cores this process may use,
# at most 16 (one GPU's share of the host)
CPU_THREADS_MAX = 16


def cpu_baseline(cfg, inp, min_seconds: float, combine: str, step_bytes: int) -> dict:
    """The oracle, unchanged, on the same workload: whole dispatch + combine
    steps until min_seconds of work (at least one), single-threaded, then the
    same with each stage split over P threads by logical rank (or expert)
    ranges, P = the cores this process may use, at most 16.  Both legs report
    µs per step and the effective GB/s of the step's algorithmic bytes."""
    from concurrent.futures import ThreadPoolExecutor

    import oracle
    fp8 = cfg.dtype == "fp8"
    d0 = oracle.run_dispatch(inp["x"], inp["idx"], cfg.E, fp8=fp8)
    y = oracle.expert_standin(d0["expert_x"], d0["expert_scale"], d0["eoff"], cfg.H)
    del d0

    def one(dispatch, combine_fn, partial_fn):
        d = dispatch()
        if combine == "partial":
            partial_fn(d)
        else:
            combine_fn(d)

    def timed(run, budget):
        steps, t0 = 0, time.perf_counter()
        while True:
            run()
            steps += 1
            el = time.perf_counter() - t0
            if el >= budget:
                return steps, el

    n1, el1 = timed(lambda: one(
        lambda: oracle.run_dispatch(inp["x"], inp["idx"], cfg.E, fp8=fp8),
        lambda d: oracle.run_combine(y, inp["w"], d, cfg.H),
        lambda d: oracle.run_partial_combine(y, inp["w"], inp["idx"], d, cfg.H)), min_seconds)
    P = max(1, min(CPU_THREADS_MAX, len(os.sched_getaffinity(0))))
    with ThreadPoolExecutor(P) as pool:
        nP, elP = timed(lambda: one(
            lambda: oracle.run_dispatch_threads(inp["x"], inp["idx"], cfg.E, P, fp8=fp8,
                                                pool=pool),
            lambda d: oracle.run_combine_threads(y, inp["w"], d, cfg.H, P, pool=pool),
            lambda d: oracle.run_partial_combine_threads(y, inp["w"], inp["idx"], d, cfg.H, P,
                                                         pool=pool)), min_seconds / 2)
    us1, usP = el1 / n1 * 1e6, elP / nP * 1e6
    cpu = host_cpu()
    return {"value": round(us1, 1), "unit": "us per dispatch+combine", "cores": 1,
            "kind": "oracle", "gbps_eff": round(step_bytes / (us1 * 1e-6) / 1e9, 3),
            "cpu_model": cpu.get("model_name", "unknown"), "host": cpu,
            "sample": f"{n1} full dispatch+combine step(s) of the {cfg.name} workload "
                      f"({cfg.N}x{cfg.T} tokens, {combine} combine), single thread, {el1:.1f} s",
            "threaded": {"value": round(usP, 1), "unit": "us per dispatch+combine", "cores": P,
                         "gbps_eff": round(step_bytes / (usP * 1e-6) / 1e9, 3),
                         "sample": f"{nP} step(s), each stage split over {P} threads by "
                                   f"logical-rank (or expert) ranges, {elP:.1f} s"}}


def main() -> int:
    ap = argparse.ArgumentParser()
    ap.add_argument("--gpus", type=int, default=1)
    # the timing protocol: 20 warmup steps, 200 timed (20 on the prefill shape)
    ap.add_argument("--steps", type=int, default=None)
    ap.add_argument("--warmup", type=int, default=20)
    ap.add_argument("--config", default="C",
                    help="workload: key (A, B, C, D, E, Ep) or name (e.g. deepseek-r1-decode)")
    ap.add_argument("--tokens", type=int, default=None,
                    help="tokens per rank (default: the workload's own)")
    ap.add_argument("--transport", choices=["staged", "direct"], default="staged",
                    help="staged: send buffer + modelled transfer (the measured contract); "
                         "direct: pack/combine write the peer's rows")
    ap.add_argument("--layout", choices=["packed", "fixed"], default="packed",
                    help="receive layout: packed at exchanged offsets, or fixed slots per "
                         "(source, local expert)")
    ap.add_argument("--combine", choices=["receiver", "partial"], default="receiver",
                    help="receiver: the token owner sums all K expert rows; partial: each "
                         "expert owner returns one pre-summed row per (token, rank)")
    ap.add_argument("--cpu-seconds", type=float, default=12.0)
    ap.add_argument("--no-cpu-baseline", action="store_true")
    ap.add_argument("--no-kernel-timing", action="store_true",
                    help="also time the steps once without per-kernel events (printed to stderr)")
    ap.add_argument("--copy-calibration", action="store_true",
                    help="run only the plain copy used to scale HBM counters")
    ap.add_argument("--traffic-from", nargs=4, metavar=("FETCH_DB", "WRITE_DB", "CAL_FETCH_DB",
                                                        "CAL_WRITE_DB"),
                    help="write profiles/traffic_<config>.json from rocprofv3 --pmc databases")
    ap.add_argument("--graph", action="store_true",
                    help="also time the step captured once as a HIP graph and replayed")
    ap.add_argument("--overlap", action="store_true",
                    help="measure the send/recv split hiding a concurrent GEMM (prints one JSON line)")
    ap.add_argument("--layer", action="store_true",
                    help="time a whole expert layer on the workload's tokens, operator by operator "
                         "(prints one JSON line)")
    ap.add_argument("--expert-width", type=int, default=2048,
                    help="with --layer: the experts' inner width (a multiple of 128)")
    ap.add_argument("--trace-summary", metavar="DB",
                    help="print a table of the library's kernels from a rocprofv3 kernel trace")
    ap.add_argument("--trace-timed", action="store_true",
                    help="with --trace-summary: add each kernel's average over the timed region "
                         "of a traced bench command run with these --steps / --warmup")
    ap.add_argument("--traffic-xcheck", nargs=5, metavar=("DRAM_DB", "CAL_DRAM_DB", "REQ_DB",
                                                          "CAL_REQ_DB", "TRAFFIC_JSON"),
                    help="print the HBM bytes per kernel from the DRAM and EA request counters "
                         "beside the FETCH_SIZE/WRITE_SIZE figures of TRAFFIC_JSON")
    args = ap.parse_args()
    from workloads import CONFIGS as _configs
    if args.config not in _configs:
        # a workload may also be named by its name ("deepseek-r1-decode", ...)
        by_name = {c.name: k for k, c in _configs.items()}
        if args.config not in by_name:
            print(f"unknown workload {args.config!r}; known: "
                  + ", ".join(f"{k} ({c.name})" for k, c in _configs.items()), file=sys.stderr)
            return 2
        args.config = by_name[args.config]
    if args.steps is None:
        args.steps = 20 if args.config == "D" else 200
    if args.copy_calibration:
        return copy_calibration()
    if args.overlap:
        from workloads import CONFIGS
        print(json.dumps(overlap_demo(CONFIGS[args.config], args)), flush=True)
        return 0
    if args.layer:
        from workloads import CONFIGS
        print(json.dumps(layer_run(CONFIGS[args.config], args)), flush=True)
        return 0
    if args.traffic_from or args.trace_summary or args.traffic_xcheck:
        from workloads import CONFIGS
        cfg = CONFIGS[args.config]
        if args.trace_summary:
            print(trace_summary(cfg, args.trace_summary,
                                (args.steps, args.warmup) if args.trace_timed else None,
                                args.layout))
        if args.traffic_xcheck:
            print(json.dumps(traffic_xcheck(cfg, *args.traffic_xcheck), indent=1))
        if args.traffic_from:
            rec = traffic_from(cfg, *args.traffic_from, transport=args.transport,
                               combine=args.combine)
            path = os.path.join(ROOT, "profiles", f"traffic_{traffic_key(args)}.json")
            with open(path, "w") as f:
                json.dump(rec, f, indent=1)
            print(json.dumps(rec, indent=1))
        return 0
    if args.gpus != 1:
        print(f"bench.py measures one GPU: the N logical ranks of the group all live on a "
              f"single device; --gpus {args.gpus} is not supported", file=sys.stderr)
        return 2

    import numpy as np
    import torch

    import combine_moe_dispatch_amd as mep
    from workloads import CONFIGS, make_inputs

    cfg = CONFIGS[args.config]
    if args.tokens is not None:
        cfg = cfg.with_(T=args.tokens)
    N, T, K, E, H = cfg.N, cfg.T, cfg.K, cfg.E, cfg.H
    R = cfg.rows
    fp8 = cfg.dtype == "fp8"
    print(f"[bench] {cfg.describe()} rows={R}", file=sys.stderr, flush=True)
    inp = make_inputs(cfg)
    dev = torch.device("cuda", 0)
    torch.cuda.set_device(dev)
    x = torch.from_numpy(inp["x"].view(np.int16)).to(dev)
    idx = torch.from_numpy(inp["idx"]).to(dev)
    w = torch.from_numpy(inp["w"]).to(dev)
    payload = H if fp8 else 2 * H
    expert_x = torch.empty((R, payload), dtype=torch.uint8, device=dev)
    expert_scale = torch.empty((R, H // 128), dtype=torch.float32, device=dev) if fp8 else None
    offs = torch.empty((E + 1,), dtype=torch.int32, device=dev)
    out = torch.empty((N, T, H), dtype=torch.bfloat16, device=dev)
    transport = mep.MOE_TRANSPORT_DIRECT if args.transport == "direct" else mep.MOE_TRANSPORT_STAGED
    partial = args.combine == "partial"
    g = mep.moe_group_create(N, E, K, H, T, mep.MOE_FP8_E4M3 if fp8 else mep.MOE_BF16, transport,
                             mep.MOE_COMBINE_PARTIAL if partial else mep.MOE_COMBINE_RECEIVER,
                             mep.MOE_LAYOUT_FIXED_SLOT if args.layout == "fixed"
                             else mep.MOE_LAYOUT_PACKED)
    stream = torch.cuda.current_stream()
    w_send = w if partial else None          # partial combine: weights go with dispatch

    # first cycle + the stand-in expert output reused by every step
    mep.moe_dispatch_send(g, T, x, idx, w_send, stream=stream)
    mep.moe_dispatch_recv(g, expert_x, expert_scale, offs, stream=stream)
    from workloads.expert import standin_expert
    y = standin_expert(torch, expert_x.view(-1), expert_scale.view(-1) if fp8 else None, offs,
                       E, H, fp8).contiguous()
    mep.moe_combine_send(g, y, stream=stream)
    mep.moe_combine_recv(g, w, out, stream=stream)
    torch.cuda.synchronize()
    assert mep.moe_group_status(g, stream) == mep.MOE_OK

    def step():
        mep.moe_dispatch_send(g, T, x, idx, w_send, stream=stream)
        mep.moe_dispatch_recv(g, expert_x, expert_scale, offs, stream=stream)
        mep.moe_combine_send(g, y, stream=stream)
        mep.moe_combine_recv(g, w, out, stream=stream)

    for _ in range(args.warmup):
        step()
    torch.cuda.synchronize()
    # per-kernel durations: an untimed pass with every kernel carrying events
    mep.moe_group_timing_enable(g, True)
    for _ in range(max(10, args.warmup)):
        step()
    timing_all = mep.moe_group_timing_read(g)
    mep.moe_group_timing_enable(g, False)
    dom = max((k for k in timing_all if timing_all[k][1]), key=lambda k: timing_all[k][0])
    # warm leg, beside the headline: the steps back to back, wall clock, no
    # kernel carrying events
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for _ in range(args.steps):
        step()
    torch.cuda.synchronize()
    warm_ms = (time.perf_counter() - t0) / args.steps * 1e3
    # timed region (the headline): each step starts with the MALL flushed (a
    # 512 MB buffer written first) and is bracketed by events; value = the
    # median step.  Only the dominant kernel carries its own events (a few us
    # per timed kernel), so its duration is measured live over exactly these
    # steps
    flush = 512 << 20
    mep.moe_group_timing_enable(g, [dom])
    torch.cuda.synchronize()
    t1 = time.perf_counter()
    cold = step_distribution(torch, step, stream, args.steps, flush_bytes=flush)
    torch.cuda.synchronize()
    t2 = time.perf_counter()
    timing_dom = mep.moe_group_timing_read(g)
    mep.moe_group_timing_enable(g, False)
    if args.no_kernel_timing:
        t3 = time.perf_counter()
        for _ in range(args.steps):
            step()
        torch.cuda.synchronize()
        print(json.dumps({"us_per_step_without_events": round((time.perf_counter() - t3) / args.steps * 1e6, 1)}),
              file=sys.stderr, flush=True)
    dist = {"cold": cold, "warm": step_distribution(torch, step, stream, args.steps),
            "flush_bytes": flush,
            "cold_wall_ms_per_step_with_flush": round((t2 - t1) / args.steps * 1e3, 4)}
    graph_rec = None
    if args.graph:
        # the four calls of one step captured as a HIP graph, then replayed:
        # the same kernels without the per-launch host work
        cap = torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.stream(cap):
            with torch.cuda.graph(graph, stream=cap):
                mep.moe_dispatch_send(g, T, x, idx, w_send, stream=cap)
                mep.moe_dispatch_recv(g, expert_x, expert_scale, offs, stream=cap)
                mep.moe_combine_send(g, y, stream=cap)
                mep.moe_combine_recv(g, w, out, stream=cap)
        for _ in range(args.warmup):
            graph.replay()
        torch.cuda.synchronize()
        t2 = time.perf_counter()
        for _ in range(args.steps):
            graph.replay()
        torch.cuda.synchronize()
        graph_rec = {"us_per_step": round((time.perf_counter() - t2) / args.steps * 1e6, 1),
                     "replays": args.steps}
        del graph
    assert mep.moe_group_status(g, stream) == mep.MOE_OK
    mep.moe_group_destroy(g)
    # the probe's source and destination each the size of one side of the
    # dominant kernel's traffic
    kb_dom = kernel_bytes(cfg, args.transport, args.combine,
                          partial_rows(cfg, inp["idx"]) if partial else 0, args.layout)[dom]
    ceiling = {"at_kernel_footprint": hbm_ceiling(torch, mep, kb_dom // 2),
               "at_1gib": hbm_ceiling(torch, mep, 1 << 30)}

    ms_per_step = cold["p50"] * 1e-3
    P = partial_rows(cfg, inp["idx"]) if partial else 0
    kb = kernel_bytes(cfg, args.transport, args.combine, P, args.layout)
    total_bytes = sum(kb.values())
    kern = {}
    for name, (ms, n) in timing_all.items():
        if n:
            avg_us = ms / n * 1e3
            kern[name] = {"avg_us": round(avg_us, 2), "launches": n,
                          "gbps": round(kb[name] / (avg_us * 1e-6) / 1e9, 1)}
    dom_ms, dom_n = timing_dom[dom]
    dom_us = dom_ms / dom_n * 1e3
    ach = kb[dom] / (dom_us * 1e-6) / 1e9
    src_hash = kernel_source_hash()
    traffic = measured_traffic(traffic_key(args), dom, src_hash)
    gbps_eff = total_bytes / (ms_per_step * 1e-3) / 1e9
    rec = {
        "metric": METRIC,
        "value": round(ms_per_step * 1e3, 1),
        "unit": "us",
        "n_gpus": 1,
        "steps": args.steps,
        "warmup": args.warmup,
        "ms_per_step": round(ms_per_step, 4),
        "higher_is_better": False,
        "scaling": "weak",
        "vs_baseline": None,
        "dtype": "fp8+bf16" if fp8 else "bf16",
        "data": "synthetic",
        "config": {"workload": cfg.describe(), "logical_ranks": N, "tokens_per_rank": T,
                   "hidden": H, "experts": E, "top_k": K, "rows": R,
                   "dispatch_dtype": cfg.dtype, "combine_dtype": "bf16",
                   "transport": args.transport, "combine": args.combine, "layout": args.layout,
                   **({"partial_rows": P} if partial else {}),
                   "parallelism": f"ep{N} (logical ranks on one GPU)"},
        "timing": "value = median of the timed steps, each started with the MALL flushed",
        "hbm_gbps_eff": round(gbps_eff, 1),
        "frac_of_hbm_peak": round(gbps_eff / HBM_PEAK_GBPS, 4),
        "warm": {"us_per_step": round(warm_ms * 1e3, 1),
                 "hbm_gbps_eff": round(total_bytes / (warm_ms * 1e-3) / 1e9, 1),
                 "frac_of_hbm_peak": round(total_bytes / (warm_ms * 1e-3) / 1e9 / HBM_PEAK_GBPS, 4),
                 "how": "wall clock over the same number of steps back to back, no flush"},
        "algorithmic_bytes_per_step": total_bytes,
        "roofline": {"bound": "hbm", "kernel": dom, "achieved": round(ach, 1),
                     "peak": HBM_PEAK_GBPS, "unit": "GB/s", "frac": round(ach / HBM_PEAK_GBPS, 4),
                     "bytes_per_launch": kb[dom], "avg_us": round(dom_us, 2),
                     "launches_timed": dom_n, "traffic": traffic,
                     "frac_of_copy_ceiling": round(
                         ach / ceiling["at_kernel_footprint"]["copy_gbps"], 4)},
        "hbm_ceiling": ceiling,
        "step_us": dist,
        "kernels": kern,
        "source_hash": src_hash,
    }
    if graph_rec is not None:
        rec["graph"] = graph_rec
    if not args.no_cpu_baseline:
        print("[bench] timing the CPU oracle", file=sys.stderr, flush=True)
        rec["cpu_baseline"] = cpu_baseline(cfg, inp, args.cpu_seconds, args.combine, total_bytes)
    else:
        rec["cpu_baseline"] = None
    print(json.dumps(rec), flush=True)
    return 0


if __name__ == "__main__":
    sys.exit(main())
