"""Python binding of libgs_splat_gb300 (include/gs_splat.h, include/gs_head.h).

Argument marshalling only: every function hands torch CUDA tensors' device
pointers and the current stream to the C entry point of the same name, and
allocates what the C call needs (outputs and workspace) with torch.  Every
step of the path runs in the library's kernels.  There is no CPU fallback:
if the library is missing or no GPU is present, calls raise.
"""

from __future__ import annotations

import contextlib
import ctypes as ct
import functools
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgs_splat_gb300.so")
LIB_DEBUG_PATH = os.path.join(_HERE, "libgs_splat_gb300_debug.so")

GS_OK = 0
STATUS_NAMES = {
    0: "GS_OK", 1: "GS_ERR_INVALID_ARG", 2: "GS_ERR_CAPACITY", 3: "GS_ERR_KEY_OUT_OF_GRID",
    4: "GS_ERR_WORKSPACE", 5: "GS_ERR_TIMEOUT", 6: "GS_ERR_CUDA", 7: "GS_ERR_UNSORTED",
    8: "GS_ERR_COUNT_MISMATCH", 9: "GS_ERR_OUT_OF_BOUNDS",
}

# exported symbol -> (restype, argtypes); mirrors include/gs_splat.h
P, I32, I64, F32, SZ = ct.c_void_p, ct.c_int, ct.c_int64, ct.c_float, ct.c_size_t
SIGNATURES = {
    "gs_version": (I32, []),
    "gs_status_string": (ct.c_char_p, [I32]),
    "gs_tile_bits": (I32, [I32, I32]),
    "gs_isect_workspace_size": (SZ, [I32, I32, I32, I32, I64, I32]),
    "gs_isect_tiles": (I32, [P, P, I32, P, I32, I32, I32, I32, I32, I32, P, P, P, P, I64, P, SZ,
                             P, P]),
    "gs_tile_offsets": (I32, [P, I64, I32, I32, I32, P, P, P]),
    "gs_rasterize_fwd": (I32, [P, P, P, P, P, P, I32, I32, I32, I32, I32, I32, P, P, I64, F32,
                               F32, P, P, P, P, P, P, P]),
    "gs_rasterize_bwd": (I32, [P, P, P, P, P, P, I32, I32, I32, I32, I32, I32, P, P, I64, F32,
                               P, P, P, P, P, P, P, P, P, P, P, P, P]),
    "gs_project": (I32, [P, P, P, P, I32, I32, I32, I32, F32, F32, F32, F32, I32, P, P, P, P, P,
                         P, P, P]),
    "gs_bin_splats": (I32, [P, P, I32, P, I32, I32, I32, I32, I32, I32, P, P, P, P]),
    "gs_rasterize_fwd_bins": (I32, [P, P, P, P, P, P, I32, I32, I32, I32, I32, I32, P, P, I32,
                                    F32, F32, P, P, P, P, P, P, P]),
    "gs_rasterize_bwd_bins": (I32, [P, P, P, P, P, P, I32, I32, I32, I32, I32, I32, P, P, I32,
                                    F32, P, P, P, P, P, P, P, P, P, P, P, P, P]),
    "gs_sort_workspace_size": (SZ, [I64]),
    "gs_sort_pairs": (I32, [P, P, I64, I32, I32, P, SZ, P, P]),
    "gs_sort_pairs_noalloc": (I32, [P, P, I64, I32, I32, P, P]),
    "gs_debug_sort_wait_timeout": (I32, [P, P, I64, I32, I32, P, SZ, P, P]),
    "gs_peak_probe": (I32, [I32, I32, I32, P, P, P]),
    "gs_rasterize_fwd_steps": (I32, [P, P, P, P, P, P, I32, I32, I32, I32, I32, I32, P, P, I64,
                                     F32, F32, I32, P, P, P, P, P, P, P, P]),
    "gs_rasterize_bwd_steps": (I32, [P, P, P, P, P, P, I32, I32, I32, I32, I32, I32, P, P, I64,
                                     F32, P, P, I32, P, P, P, P, P, P, P, P, P, P, P, P, P]),
    "gs_layer_norm_fwd": (I32, [P, I64, P, P, I64, I32, I32, I32, F32, P, I64, P, P, P]),
    "gs_layer_norm_bwd_workspace_size": (SZ, [I64, I32]),
    "gs_layer_norm_bwd": (I32, [P, I64, P, I64, P, P, P, I64, I32, I32, I32, P, I64, P, P, P, SZ,
                                P]),
    "gs_expert_sort_workspace_size": (SZ, [I64, I32, I32]),
    "gs_expert_sort": (I32, [P, I64, I32, I32, P, P, P, P, SZ, P]),
    "gs_expert_dispatch": (I32, [P, I64, P, P, I64, I32, I32, I32, I32, P, P, P]),
    "gs_expert_combine": (I32, [P, P, P, I64, I32, I32, I32, P, I64, P, P]),
    "gs_expert_combine_bwd": (I32, [P, I64, P, P, P, P, I64, I32, I32, I32, I32, P, P, P, P]),
    "gs_expert_linear_fwd_workspace_size": (SZ, [I64, I32, I32, I32, I32, I32]),
    "gs_expert_linear_fwd": (I32, [P, P, P, P, I64, I32, I32, I32, I32, P, P, SZ, P, P]),
    "gs_expert_linear_bwd_workspace_size": (SZ, [I64, I32, I32, I32, I32, I32]),
    "gs_expert_linear_bwd": (I32, [P, P, P, P, I64, I32, I32, I32, I32, P, P, P, P, SZ, P, P]),
    "gs_expert_route_workspace_size": (SZ, [I64, I32]),
    "gs_expert_route_fwd": (I32, [P, I64, P, I64, I32, I32, I32, I32, P, P, P, P, P, SZ, P]),
    "gs_expert_route_bwd": (I32, [P, I64, P, P, P, P, I64, I32, I32, I32, I32, P, I64, P, P]),
    "gs_rows_pack8": (I32, [P, I64, I64, I32, I32, P, P, P]),
    "gs_rows_unpack8": (I32, [P, P, I64, I32, I32, P, I64, P]),
    "gs_expert_linear8_fwd": (I32, [P, P, P, P, P, P, I64, I32, I32, I32, I32, P, P, P]),
    "gs_expert_linear8_bwd_workspace_size": (SZ, [I64, I32, I32, I32, I32, I32]),
    "gs_expert_linear8_bwd": (I32, [P, P, P, P, P, P, I64, I32, I32, I32, I32, P, P, P, P, SZ, P,
                                    P]),
}


class GsError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {STATUS_NAMES.get(code, code)} ({_status_text(code)})")


_lib = None


def _load(path):
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: build it with `python -c 'import __graft_entry__ as g; "
            "g.build()'` (the CUDA library has no CPU fallback)")
    L = ct.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    return L


def lib():
    """Opens the library (once).  Raises if it was not built."""
    global _lib
    if _lib is None:
        _lib = _load(LIB_PATH)
    return _lib


@contextlib.contextmanager
def library(path):
    """Routes this module's calls to another build of the library -- the
    range-checking build, LIB_DEBUG_PATH -- while the block runs."""
    global _lib
    saved = _lib
    _lib = _load(path)
    try:
        yield _lib
    finally:
        _lib = saved


def _status_text(code):
    try:
        return lib().gs_status_string(code).decode()
    except Exception:  # pragma: no cover
        return "?"


def _check(code, where):
    if code != GS_OK:
        raise GsError(code, where)


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr() or None


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _empty(shape, dtype, device):
    return torch.empty(shape, dtype=dtype, device=device)


def new_status(device) -> torch.Tensor:
    return torch.zeros(1, dtype=torch.int32, device=device)


def check_status(d_status: torch.Tensor, where: str = "device"):
    """Reads a device status word (synchronises) and raises on an error."""
    code = int(d_status.item())
    _check(code, where)


def gs_tile_bits(tile_width: int, tile_height: int) -> int:
    return int(lib().gs_tile_bits(tile_width, tile_height))


def gs_isect_workspace_size(C, N, tile_width, tile_height, n_isects, sort=True) -> int:
    return int(lib().gs_isect_workspace_size(C, N, tile_width, tile_height, n_isects, int(sort)))


def gs_isect_tiles(means2d, radii, depths, tile_size, tile_width, tile_height, sort=True,
                   d_status=None, workspace=None, stream=None):
    """Both calls of the C entry point: the size query, then the emission.
    Returns (tiles_per_gauss (C,N) int32, keys (I,) int64 holding the uint64
    bits, flatten_ids (I,) int32)."""
    C, N = means2d.shape[:2]
    dev = means2d.device
    ell = int(radii.dim() == 3)
    tpg = _empty((C, N), torch.int32, dev)
    s = _stream(stream)
    q_bytes = gs_isect_workspace_size(C, N, tile_width, tile_height, 0, sort)
    ws = workspace if workspace is not None and workspace.numel() >= q_bytes else \
        _empty(q_bytes, torch.uint8, dev)
    total = ct.c_int64(0)
    _check(lib().gs_isect_tiles(_ptr(means2d), _ptr(radii), ell, _ptr(depths), C, N, tile_size,
                                tile_width, tile_height, int(sort), _ptr(tpg), ct.byref(total),
                                None, None, 0, _ptr(ws), ws.numel(), _ptr(d_status), s),
           "gs_isect_tiles (size query)")
    I = int(total.value)
    keys = _empty(I, torch.int64, dev)
    ids = _empty(I, torch.int32, dev)
    if I == 0:
        return tpg, keys, ids
    e_bytes = gs_isect_workspace_size(C, N, tile_width, tile_height, I, sort)
    if ws.numel() < e_bytes:
        ws = _empty(e_bytes, torch.uint8, dev)
    _check(lib().gs_isect_tiles(_ptr(means2d), _ptr(radii), ell, _ptr(depths), C, N, tile_size,
                                tile_width, tile_height, int(sort), None, None, _ptr(keys),
                                _ptr(ids), I, _ptr(ws), ws.numel(), _ptr(d_status), s),
           "gs_isect_tiles")
    return tpg, keys, ids


def gs_tile_offsets(keys, C, tile_width, tile_height, d_status=None, out=None, stream=None):
    """offsets (C, tile_height, tile_width) int32 from sorted keys."""
    offsets = out if out is not None else _empty((C, tile_height, tile_width), torch.int32,
                                                 keys.device)
    _check(lib().gs_tile_offsets(_ptr(keys), keys.numel(), C, tile_width, tile_height,
                                 _ptr(offsets), _ptr(d_status), _stream(stream)),
           "gs_tile_offsets")
    return offsets


def gs_project(means, covars, viewmats, intrinsics, width, height, eps2d=0.3, near_plane=0.01,
               far_plane=1e10, radius_clip=0.0, compensation=False, orthographic=False,
               radii_float=False, d_status=None, out=None, stream=None):
    """EWA projection.  means (N,3), covars (N,3,3), viewmats (C,4,4),
    intrinsics (C,3,3), float32 CUDA tensors.  Returns dict(radii int32
    (C,N,2), means2d (C,N,2), depths (C,N), conics (C,N,3), compensations
    (C,N) or None, radii_float (C,N,2) or None: the radii as gs_isect_tiles
    takes them)."""
    N = means.shape[0]
    C = viewmats.shape[0]
    dev = means.device
    if out is None:
        out = dict(radii=_empty((C, N, 2), torch.int32, dev),
                   means2d=_empty((C, N, 2), torch.float32, dev),
                   depths=_empty((C, N), torch.float32, dev),
                   conics=_empty((C, N, 3), torch.float32, dev),
                   compensations=_empty((C, N), torch.float32, dev) if compensation else None,
                   radii_float=_empty((C, N, 2), torch.float32, dev) if radii_float else None)
    _check(lib().gs_project(
        _ptr(means), _ptr(covars), _ptr(viewmats), _ptr(intrinsics), C, N, int(width),
        int(height), float(eps2d), float(near_plane), float(far_plane), float(radius_clip),
        int(bool(orthographic)), _ptr(out["radii"]), _ptr(out["means2d"]), _ptr(out["depths"]),
        _ptr(out["conics"]), _ptr(out["compensations"]), _ptr(out["radii_float"]),
        _ptr(d_status), _stream(stream)), "gs_project")
    return out


def gs_bin_splats(means2d, radii, depths, tile_size, tile_width, tile_height, capacity,
                  d_status=None, out=None, stream=None):
    """Returns (bins int32 (C, TH, TW, capacity) with -1 after each bin's
    splats, bin_counts int32 (C, TH, TW))."""
    C, N = means2d.shape[:2]
    dev = means2d.device
    if out is None:
        out = (_empty((C, tile_height, tile_width, capacity), torch.int32, dev),
               _empty((C, tile_height, tile_width), torch.int32, dev))
    bins, counts = out
    _check(lib().gs_bin_splats(
        _ptr(means2d), _ptr(radii), int(radii.dim() == 3), _ptr(depths), C, N, tile_size,
        tile_width, tile_height, int(capacity), _ptr(bins), _ptr(counts), _ptr(d_status),
        _stream(stream)), "gs_bin_splats")
    return bins, counts


def gs_rasterize_fwd(means2d, conics, colors, opacities, backgrounds, masks, width, height,
                     tile_size, offsets, flatten_ids, alpha_cutoff, transmittance_threshold,
                     d_status=None, out=None, pair_counts=None, trace=None, stream=None):
    """Returns (render_colors (C,H,W,ch), render_alphas (C,H,W,1), last_ids (C,H,W)).
    pair_counts: optional int32 (C,H,W,3) tensor that receives per pixel the
    entries evaluated, the entries composited and the entries evaluated up
    to the last composited one.  trace: optional int32 (n_isects, 8) tensor
    that receives the per-entry composite masks for gs_rasterize_bwd."""
    C, N = means2d.shape[:2]
    ch = colors.shape[-1]
    dev = means2d.device
    if out is None:
        out = (_empty((C, height, width, ch), torch.float32, dev),
               _empty((C, height, width, 1), torch.float32, dev),
               _empty((C, height, width), torch.int32, dev))
    rgb, alpha, last = out
    _check(lib().gs_rasterize_fwd(
        _ptr(means2d), _ptr(conics), _ptr(colors), _ptr(opacities), _ptr(backgrounds),
        _ptr(masks), C, N, ch, width, height, tile_size, _ptr(offsets), _ptr(flatten_ids),
        flatten_ids.numel(), float(alpha_cutoff), float(transmittance_threshold), _ptr(rgb),
        _ptr(alpha), _ptr(last), _ptr(pair_counts), _ptr(trace), _ptr(d_status),
        _stream(stream)), "gs_rasterize_fwd")
    return rgb, alpha, last


def gs_rasterize_bwd(means2d, conics, colors, opacities, backgrounds, masks, width, height,
                     tile_size, offsets, flatten_ids, alpha_cutoff, render_alphas, last_ids,
                     grad_render_colors, grad_render_alphas, want_grad_backgrounds=None,
                     absgrad=False, d_status=None, out=None, trace=None, stream=None):
    """Returns dict(grad_means2d, grad_conics, grad_colors, grad_opacities,
    grad_backgrounds (or None), grad_means2d_abs (or None)).  trace: the mask
    table the forward wrote for the same inputs (optional, faster)."""
    C, N = means2d.shape[:2]
    ch = colors.shape[-1]
    dev = means2d.device
    if want_grad_backgrounds is None:
        want_grad_backgrounds = backgrounds is not None
    if out is None:
        out = dict(grad_means2d=_empty((C, N, 2), torch.float32, dev),
                   grad_conics=_empty((C, N, 3), torch.float32, dev),
                   grad_colors=_empty((C, N, ch), torch.float32, dev),
                   grad_opacities=_empty((C, N), torch.float32, dev),
                   grad_backgrounds=_empty((C, ch), torch.float32, dev)
                   if want_grad_backgrounds else None,
                   grad_means2d_abs=_empty((C, N, 2), torch.float32, dev) if absgrad else None)
    _check(lib().gs_rasterize_bwd(
        _ptr(means2d), _ptr(conics), _ptr(colors), _ptr(opacities), _ptr(backgrounds),
        _ptr(masks), C, N, ch, width, height, tile_size, _ptr(offsets), _ptr(flatten_ids),
        flatten_ids.numel(), float(alpha_cutoff), _ptr(render_alphas), _ptr(last_ids),
        _ptr(grad_render_colors), _ptr(grad_render_alphas), _ptr(out["grad_means2d"]),
        _ptr(out["grad_conics"]), _ptr(out["grad_colors"]), _ptr(out["grad_opacities"]),
        _ptr(out["grad_backgrounds"]), _ptr(out["grad_means2d_abs"]), _ptr(trace),
        _ptr(d_status), _stream(stream)), "gs_rasterize_bwd")
    return out


def gs_sort_pairs(keys, values, begin_bit=0, end_bit=64, d_status=None, workspace=None,
                  stream=None):
    """Stable in-place sort of (keys int64 holding uint64 bits, values int32)
    by key bits [begin_bit, end_bit)."""
    n = keys.numel()
    need = int(lib().gs_sort_workspace_size(n))
    ws = workspace if workspace is not None and workspace.numel() >= need else \
        _empty(max(need, 1), torch.uint8, keys.device)
    _check(lib().gs_sort_pairs(_ptr(keys), _ptr(values), n, begin_bit, end_bit, _ptr(ws),
                               ws.numel(), _ptr(d_status), _stream(stream)), "gs_sort_pairs")
    return keys, values


SORT_NOALLOC_MAX_PAIRS = 1 << 20


def gs_sort_pairs_noalloc(keys, values, begin_bit=0, end_bit=64, d_status=None, stream=None):
    """gs_sort_pairs without a workspace: the library's own fixed scratch
    array is used (n <= SORT_NOALLOC_MAX_PAIRS; calls on one device must not
    overlap on the GPU)."""
    _check(lib().gs_sort_pairs_noalloc(_ptr(keys), _ptr(values), keys.numel(), begin_bit,
                                       end_bit, _ptr(d_status), _stream(stream)),
           "gs_sort_pairs_noalloc")
    return keys, values


def gs_rasterize_fwd_bins(means2d, conics, colors, opacities, backgrounds, masks, width, height,
                          tile_size, bins, bin_counts, alpha_cutoff, transmittance_threshold,
                          d_status=None, out=None, pair_counts=None, trace=None, stream=None):
    """gs_rasterize_fwd over bin lists (bins (C, TH, TW, M), bin_counts).
    last_ids and trace rows are positions in bins."""
    C, N = means2d.shape[:2]
    ch = colors.shape[-1]
    dev = means2d.device
    if out is None:
        out = (_empty((C, height, width, ch), torch.float32, dev),
               _empty((C, height, width, 1), torch.float32, dev),
               _empty((C, height, width), torch.int32, dev))
    rgb, alpha, last = out
    _check(lib().gs_rasterize_fwd_bins(
        _ptr(means2d), _ptr(conics), _ptr(colors), _ptr(opacities), _ptr(backgrounds),
        _ptr(masks), C, N, ch, width, height, tile_size, _ptr(bins), _ptr(bin_counts),
        bins.shape[-1], float(alpha_cutoff), float(transmittance_threshold), _ptr(rgb),
        _ptr(alpha), _ptr(last), _ptr(pair_counts), _ptr(trace), _ptr(d_status),
        _stream(stream)), "gs_rasterize_fwd_bins")
    return rgb, alpha, last


def gs_rasterize_bwd_bins(means2d, conics, colors, opacities, backgrounds, masks, width, height,
                          tile_size, bins, bin_counts, alpha_cutoff, render_alphas, last_ids,
                          grad_render_colors, grad_render_alphas, want_grad_backgrounds=None,
                          absgrad=False, d_status=None, out=None, trace=None, stream=None):
    """gs_rasterize_bwd over bin lists; same outputs as gs_rasterize_bwd."""
    C, N = means2d.shape[:2]
    ch = colors.shape[-1]
    dev = means2d.device
    if want_grad_backgrounds is None:
        want_grad_backgrounds = backgrounds is not None
    if out is None:
        out = dict(grad_means2d=_empty((C, N, 2), torch.float32, dev),
                   grad_conics=_empty((C, N, 3), torch.float32, dev),
                   grad_colors=_empty((C, N, ch), torch.float32, dev),
                   grad_opacities=_empty((C, N), torch.float32, dev),
                   grad_backgrounds=_empty((C, ch), torch.float32, dev)
                   if want_grad_backgrounds else None,
                   grad_means2d_abs=_empty((C, N, 2), torch.float32, dev) if absgrad else None)
    _check(lib().gs_rasterize_bwd_bins(
        _ptr(means2d), _ptr(conics), _ptr(colors), _ptr(opacities), _ptr(backgrounds),
        _ptr(masks), C, N, ch, width, height, tile_size, _ptr(bins), _ptr(bin_counts),
        bins.shape[-1], float(alpha_cutoff), _ptr(render_alphas), _ptr(last_ids),
        _ptr(grad_render_colors), _ptr(grad_render_alphas), _ptr(out["grad_means2d"]),
        _ptr(out["grad_conics"]), _ptr(out["grad_colors"]), _ptr(out["grad_opacities"]),
        _ptr(out["grad_backgrounds"]), _ptr(out["grad_means2d_abs"]), _ptr(trace),
        _ptr(d_status), _stream(stream)), "gs_rasterize_bwd_bins")
    return out


def gs_debug_sort_wait_timeout(keys, values, ticket_start, wait_polls, d_status, stream=None):
    """Test hook of the timeout path (see the header): one sorting pass whose
    first look-back word is never published and whose waits poll at most
    wait_polls times.  keys int64 (n), values int32 (n) are overwritten with
    unspecified values; d_status receives GS_ERR_TIMEOUT."""
    n = keys.numel()
    ws = _empty(lib().gs_sort_workspace_size(n + ticket_start * 2048), torch.uint8, keys.device)
    _check(lib().gs_debug_sort_wait_timeout(_ptr(keys), _ptr(values), n, ticket_start,
                                            wait_polls, _ptr(ws), ws.numel(), _ptr(d_status),
                                            _stream(stream)), "gs_debug_sort_wait_timeout")
    return ws


def gs_peak_probe(kind, iters, blocks, out, stream=None):
    """Enqueues the throughput probe (kind 0 FMA, 1 packed FMA, 2 ex2) into
    out (float32, blocks * 256); returns the number of operations."""
    ops = ct.c_int64(0)
    _check(lib().gs_peak_probe(kind, iters, blocks, _ptr(out), ct.byref(ops), _stream(stream)),
           "gs_peak_probe")
    return int(ops.value)


def gs_rasterize_fwd_steps(means2d, conics, colors, opacities, backgrounds, masks, width, height,
                           tile_size, offsets, flatten_ids, alpha_cutoff,
                           transmittance_threshold, max_steps, d_status=None, stream=None):
    """gs_rasterize_fwd that also records the per-pixel step trace.  Returns
    (render_colors, render_alphas, last_ids, (step_pos, step_T, step_count))
    with step_pos int32 / step_T float32 (max_steps, C, H, W) and step_count
    int32 (C, H, W)."""
    C, N = means2d.shape[0], means2d.shape[1]
    ch = colors.shape[-1]
    dev = means2d.device
    rgb = _empty((C, height, width, ch), torch.float32, dev)
    alpha = _empty((C, height, width, 1), torch.float32, dev)
    last = _empty((C, height, width), torch.int32, dev)
    pos = _empty((max_steps, C, height, width), torch.int32, dev)
    tb = _empty((max_steps, C, height, width), torch.float32, dev)
    cnt = _empty((C, height, width), torch.int32, dev)
    _check(lib().gs_rasterize_fwd_steps(
        _ptr(means2d), _ptr(conics), _ptr(colors), _ptr(opacities), _ptr(backgrounds),
        _ptr(masks), C, N, ch, width, height, tile_size, _ptr(offsets), _ptr(flatten_ids),
        flatten_ids.numel(), alpha_cutoff, transmittance_threshold, max_steps, _ptr(rgb),
        _ptr(alpha), _ptr(last), _ptr(pos), _ptr(tb), _ptr(cnt), _ptr(d_status),
        _stream(stream)), "gs_rasterize_fwd_steps")
    return rgb, alpha, last, (pos, tb, cnt)


def gs_rasterize_bwd_steps(means2d, conics, colors, opacities, backgrounds, masks, width, height,
                           tile_size, offsets, flatten_ids, alpha_cutoff, render_alphas,
                           last_ids, steps, grad_render_colors, grad_render_alphas,
                           absgrad=False, d_status=None, out=None, stream=None):
    """The backward over a step trace `steps` = (step_pos, step_T, step_count)
    from gs_rasterize_fwd_steps.  Returns the gradients as gs_rasterize_bwd."""
    C, N = means2d.shape[0], means2d.shape[1]
    ch = colors.shape[-1]
    dev = means2d.device
    pos, tb, cnt = steps
    if out is None:
        out = dict(grad_means2d=_empty((C, N, 2), torch.float32, dev),
                   grad_conics=_empty((C, N, 3), torch.float32, dev),
                   grad_colors=_empty((C, N, ch), torch.float32, dev),
                   grad_opacities=_empty((C, N), torch.float32, dev),
                   grad_backgrounds=None if backgrounds is None else
                   _empty((C, ch), torch.float32, dev),
                   grad_means2d_abs=_empty((C, N, 2), torch.float32, dev) if absgrad else None)
    _check(lib().gs_rasterize_bwd_steps(
        _ptr(means2d), _ptr(conics), _ptr(colors), _ptr(opacities), _ptr(backgrounds),
        _ptr(masks), C, N, ch, width, height, tile_size, _ptr(offsets), _ptr(flatten_ids),
        flatten_ids.numel(), alpha_cutoff, _ptr(render_alphas), _ptr(last_ids), pos.shape[0],
        _ptr(pos), _ptr(tb), _ptr(cnt), _ptr(grad_render_colors), _ptr(grad_render_alphas),
        _ptr(out["grad_means2d"]), _ptr(out["grad_conics"]), _ptr(out["grad_colors"]),
        _ptr(out["grad_opacities"]), _ptr(out["grad_backgrounds"]),
        _ptr(out["grad_means2d_abs"]), _ptr(d_status), _stream(stream)),
        "gs_rasterize_bwd_steps")
    return out


# ---- the feature head (include/gs_head.h) ------------------------------------
#
# A call on one token is over in a few microseconds on the GPU, so the checks
# build no message before they fail and the stream is read as its raw handle.
#
# d_status (new_status, check_status) is where the kernels report: without it a
# wait that ran out (GS_ERR_TIMEOUT) leaves part of an output unwritten and
# nothing is raised.

_DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # None: a torch without CUDA


def _dtype(t, what):
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{what}: float32, float16 or bfloat16 expected, not {t.dtype}")
    return code


def _refuse(what):
    raise ValueError(what)


def _rows(t, what):
    """(data pointer, row distance) of a (..., channels) tensor whose rows lie
    at one distance, such as a channel slice of a contiguous image."""
    if not t.is_cuda:
        _refuse(f"{what}: expected a CUDA tensor")
    if t.dim() == 0:
        _refuse(f"{what}: at least one dimension expected")
    ch = t.shape[-1]
    if t.is_contiguous():
        return t.data_ptr() or None, ch
    shape, stride = t.shape, t.stride()
    ld, rows = None, 1
    for d in range(t.dim() - 2, -1, -1):
        if shape[d] == 1:
            continue
        if ld is None:
            ld = stride[d]
        if stride[d] != ld * rows:
            _refuse(f"{what}: the rows must lie at one distance")
        rows *= shape[d]
    if ch > 1 and stride[-1] != 1:
        _refuse(f"{what}: the channels of a row must be contiguous")
    ld = ch if ld is None else ld
    if t.numel() and ld < ch:
        _refuse(f"{what}: rows must not overlap")
    return t.data_ptr() or None, ld


@functools.cache
def _devices():
    return torch.cuda.device_count()


def _on(stream, like, *others):
    """The call's stream as a raw handle: `stream`, or the current one of the
    device that `like` is on, which has to be the current device and that of
    the call's other tensors (or None)."""
    if not like.is_cuda:
        _refuse("expected a CUDA tensor")
    device = like.get_device()
    if device != torch.cuda.current_device() or \
            getattr(stream, "device_index", device) != device:
        _refuse("tensors and stream of the current device expected")
    if _devices() > 1:  # else every CUDA tensor is on the one there is
        for t in others:
            if t is not None and t.get_device() != device:
                _refuse("tensors and stream of the current device expected")
    return _raw_stream(device) if stream is None else stream.cuda_stream


def _new(shape, dtype, like, stream):
    """An output or workspace of the call, of its stream's memory: a block that
    the current stream has freed may still be in use there.  The allocator is
    told that the current stream, where the caller goes on, may use it too."""
    if stream is None or stream.cuda_stream == _raw_stream(like.get_device()):
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=like.device)
    t.record_stream(torch.cuda.current_stream(like.device))
    return t


def _workspace(workspace, n_bytes, like, stream):
    if workspace is not None and workspace.numel() * workspace.element_size() >= n_bytes:
        return workspace
    return _new((n_bytes,), torch.uint8, like, stream)


def _same(t, shape, dtype, what):
    if t.shape != shape or t.dtype != dtype:
        _refuse(f"{what}: shape {tuple(shape)} and type {dtype} expected")
    return t


def _norm_params(x, weight, bias):
    """The common type of weight and bias: float32 or x's."""
    p = weight.dtype if weight is not None else bias.dtype if bias is not None else torch.float32
    if p is not torch.float32 and p != x.dtype:
        _refuse("weight, bias: float32 or the type of x expected")
    for t in (weight, bias):
        if t is not None:
            _same(t, x.shape[-1:], p, "weight, bias")
    return p


def gs_layer_norm_fwd(x, weight=None, bias=None, eps=1e-5, out=None, stats=True, stream=None):
    """Layer norm over the last dimension of x (float32, float16 or bfloat16;
    rows may be a channel slice of a wider image).  weight, bias (channels,)
    of float32 or x's type, or None.  Returns (y, mean, rstd) with mean and
    rstd float32 of x's leading shape (None without stats)."""
    dt = _dtype(x, "x")
    xp, ldx = _rows(x, "x")
    shape = x.shape
    ch = shape[-1]
    p = _norm_params(x, weight, bias)
    if out is None:
        y = _new(shape, x.dtype, x, stream)
        yp, ldy = y.data_ptr() or None, ch
    else:
        y = _same(out, shape, x.dtype, "out")
        yp, ldy = _rows(y, "out")
    mean = rstd = None
    if stats:
        mean = _new(shape[:-1], torch.float32, x, stream)
        rstd = _new(shape[:-1], torch.float32, x, stream)
    _check(lib().gs_layer_norm_fwd(xp, ldx, _ptr(weight), _ptr(bias),
                                   x.numel() // ch if ch else 0, ch, dt, _DTYPES[p], eps, yp, ldy,
                                   _ptr(mean), _ptr(rstd), _on(stream, x, weight, bias, out)),
           "gs_layer_norm_fwd")
    return y, mean, rstd


def gs_layer_norm_bwd(grad_y, x, weight, mean, rstd, out=None, params=True, param_dtype=None,
                      workspace=None, stream=None):
    """Gradients of gs_layer_norm_fwd: (grad_x, grad_weight, grad_bias), the
    last two of weight's type (param_dtype, default float32, without a
    weight), or None without params.  out: where grad_x goes, such as the
    channel slice of a wider gradient image."""
    dt = _dtype(x, "x")
    xp, ldx = _rows(x, "x")
    shape = x.shape
    gp, ldg = _rows(_same(grad_y, shape, x.dtype, "grad_y"), "grad_y")
    ch = shape[-1]
    rows = x.numel() // ch if ch else 0
    p = _norm_params(x, weight, None) if weight is not None else param_dtype or torch.float32
    if p is not torch.float32 and p != x.dtype:
        _refuse("param_dtype: float32 or the type of x expected")
    for t in (mean, rstd):
        if t.numel() != rows or t.dtype != torch.float32:
            _refuse("mean, rstd: one float32 per row expected")
    if out is None:
        gx = _new(shape, x.dtype, x, stream)
        op, ldo = gx.data_ptr() or None, ch
    else:
        gx = _same(out, shape, x.dtype, "out")
        op, ldo = _rows(gx, "out")
    gw = gb = ws = None
    n_bytes = 0
    L = lib()
    if params:
        gw, gb = _new((ch,), p, x, stream), _new((ch,), p, x, stream)
        n_bytes = L.gs_layer_norm_bwd_workspace_size(rows, ch)
        ws = _workspace(workspace, n_bytes, x, stream)
    _check(L.gs_layer_norm_bwd(gp, ldg, xp, ldx, _ptr(weight), _ptr(mean), _ptr(rstd), rows, ch,
                               dt, _DTYPES[p], op, ldo, _ptr(gw), _ptr(gb), _ptr(ws), n_bytes,
                               _on(stream, x, grad_y, weight, mean, rstd, out, ws)),
           "gs_layer_norm_bwd")
    return gx, gw, gb


def gs_expert_sort(expert_ids, experts, workspace=None, stream=None):
    """Sorts the (token, choice) pairs of expert_ids int32 (tokens, topk) by
    expert; an id outside [0, experts) drops its pair.  Returns (offsets
    int32 (experts + 1,), order int32 (tokens * topk,), slots int32
    (tokens, topk))."""
    if expert_ids.dim() != 2 or expert_ids.dtype != torch.int32:
        _refuse("expert_ids: int32 (tokens, topk) expected")
    T, k = expert_ids.shape
    if experts < 0:
        _refuse("experts: a count expected")
    offsets = _new((experts + 1,), torch.int32, expert_ids, stream)
    order = _new((T * k,), torch.int32, expert_ids, stream)
    slots = _new((T, k), torch.int32, expert_ids, stream)
    L = lib()
    n_bytes = L.gs_expert_sort_workspace_size(T, k, experts)
    ws = _workspace(workspace, n_bytes, expert_ids, stream) if n_bytes else None
    _check(L.gs_expert_sort(_ptr(expert_ids), T, k, experts, _ptr(offsets), _ptr(order),
                            _ptr(slots), _ptr(ws), n_bytes, _on(stream, expert_ids, ws)),
           "gs_expert_sort")
    return offsets, order, slots


def _pairs(slots):
    if slots.dim() != 2 or slots.dtype != torch.int32:
        _refuse("slots: int32 (tokens, topk) expected")
    return slots.shape


def _experts(offsets):
    if offsets.dim() != 1 or offsets.numel() < 2 or offsets.dtype != torch.int32:
        _refuse("offsets: int32 (experts + 1,) expected")
    return offsets.numel() - 1


def _pair_weights(weights, slots):
    if weights is not None:
        _same(weights, slots.shape, torch.float32, "weights")
    return _ptr(weights)


def gs_expert_dispatch(x, slots, offsets, d_status=None, out=None, stream=None):
    """x's rows (tokens, channels) in expert order: (tokens * topk, channels),
    zero rows behind the kept pairs."""
    dt = _dtype(x, "x")
    T, k = _pairs(slots)
    E = _experts(offsets)
    if x.dim() != 2 or x.shape[0] != T:
        _refuse("x: (tokens, channels) expected")
    ch = x.shape[1]
    xp, ldx = _rows(x, "x")
    xs = _new((T * k, ch), x.dtype, x, stream) if out is None else \
        _same(out, (T * k, ch), x.dtype, "out")
    _check(lib().gs_expert_dispatch(xp, ldx, _ptr(slots), _ptr(offsets), T, k, E, ch, dt,
                                    _ptr(xs), _ptr(d_status),
                                    _on(stream, x, slots, offsets, d_status, out)),
           "gs_expert_dispatch")
    return xs


def gs_expert_combine(ys, slots, weights=None, d_status=None, out=None, stream=None):
    """The weighted sum of every token's rows of ys (tokens * topk, channels):
    (tokens, channels).  weights float32 (tokens, topk), None for ones (the
    gradient of gs_expert_dispatch)."""
    dt = _dtype(ys, "ys")
    T, k = _pairs(slots)
    if ys.dim() != 2 or ys.shape[0] != T * k:
        _refuse("ys: (tokens * topk, channels) expected")
    ch = ys.shape[1]
    if out is None:
        y = _new((T, ch), ys.dtype, ys, stream)
        yp, ldy = y.data_ptr() or None, ch
    else:
        y = _same(out, (T, ch), ys.dtype, "out")
        yp, ldy = _rows(y, "out")
    _check(lib().gs_expert_combine(_ptr(ys), _ptr(slots), _pair_weights(weights, slots), T, k, ch,
                                   dt, yp, ldy, _ptr(d_status),
                                   _on(stream, ys, slots, weights, d_status, out)),
           "gs_expert_combine")
    return y


def gs_expert_combine_bwd(grad_y, ys, slots, weights, offsets, d_status=None, stream=None):
    """Gradients of gs_expert_combine: (grad_ys (tokens * topk, channels),
    grad_weights float32 (tokens, topk), None without weights)."""
    dt = _dtype(ys, "ys")
    T, k = _pairs(slots)
    E = _experts(offsets)
    if ys.dim() != 2 or ys.shape[0] != T * k:
        _refuse("ys: (tokens * topk, channels) expected")
    ch = ys.shape[1]
    gp, ldg = _rows(_same(grad_y, (T, ch), ys.dtype, "grad_y"), "grad_y")
    gys = _new((T * k, ch), ys.dtype, ys, stream)
    gw = _new((T, k), torch.float32, ys, stream) if weights is not None else None
    _check(lib().gs_expert_combine_bwd(gp, ldg, _ptr(ys), _ptr(slots),
                                       _pair_weights(weights, slots), _ptr(offsets), T, k, E, ch,
                                       dt, _ptr(gys), _ptr(gw), _ptr(d_status),
                                       _on(stream, ys, grad_y, slots, weights, offsets, d_status)),
           "gs_expert_combine_bwd")
    return gys, gw


def _linear_shapes(xs, offsets, weight):
    E = _experts(offsets)
    if weight.dim() != 3 or weight.shape[0] != E or weight.dtype != xs.dtype:
        _refuse("weight: (experts, out_features, in_features) of the rows' type expected")
    _, o, i = weight.shape
    if xs.dim() != 2 or xs.shape[1] != i:
        _refuse("xs: (rows, in_features) expected")
    return E, i, o


def gs_expert_linear_fwd(xs, offsets, weight, bias=None, d_status=None, out=None, workspace=None,
                         stream=None):
    """Every expert's product over its sorted rows: xs (rows, in_features),
    weight (experts, out_features, in_features), bias (experts, out_features)
    or None.  Returns ys (rows, out_features), zero rows behind the last
    expert's."""
    dt = _dtype(xs, "xs")
    E, i, o = _linear_shapes(xs, offsets, weight)
    R = xs.shape[0]
    if bias is not None:
        _same(bias, (E, o), xs.dtype, "bias")
    ys = _new((R, o), xs.dtype, xs, stream) if out is None else \
        _same(out, (R, o), xs.dtype, "out")
    L = lib()
    aligned = (xs.data_ptr() | weight.data_ptr()) % 16 == 0
    n_bytes = L.gs_expert_linear_fwd_workspace_size(R, E, i, o, dt, aligned)
    ws = _workspace(workspace, n_bytes, xs, stream) if n_bytes else None
    _check(L.gs_expert_linear_fwd(_ptr(xs), _ptr(offsets), _ptr(weight), _ptr(bias), R, E, i, o,
                                  dt, _ptr(ys), _ptr(ws), n_bytes, _ptr(d_status),
                                  _on(stream, xs, offsets, weight, bias, d_status, out, ws)),
           "gs_expert_linear_fwd")
    return ys


def gs_expert_linear_bwd(grad_ys, xs, offsets, weight, bias=True, input=True, d_status=None,
                         workspace=None, stream=None):
    """Gradients of gs_expert_linear_fwd: (grad_xs, grad_weight, grad_bias),
    the first None without `input`, the last None without `bias`."""
    dt = _dtype(xs, "xs")
    E, i, o = _linear_shapes(xs, offsets, weight)
    R = xs.shape[0]
    _same(grad_ys, (R, o), xs.dtype, "grad_ys")
    gx = _new((R, i), xs.dtype, xs, stream) if input else None
    gw = _new((E, o, i), xs.dtype, xs, stream)
    gb = _new((E, o), xs.dtype, xs, stream) if bias else None
    L = lib()
    aligned = (grad_ys.data_ptr() | xs.data_ptr() | weight.data_ptr()) % 16 == 0
    n_bytes = L.gs_expert_linear_bwd_workspace_size(R, E, i, o, dt, aligned)
    ws = _workspace(workspace, n_bytes, xs, stream) if n_bytes else None
    _check(L.gs_expert_linear_bwd(_ptr(grad_ys), _ptr(xs), _ptr(offsets), _ptr(weight), R, E, i,
                                  o, dt, _ptr(gx), _ptr(gw), _ptr(gb), _ptr(ws), n_bytes,
                                  _ptr(d_status),
                                  _on(stream, xs, grad_ys, offsets, weight, d_status, ws)),
           "gs_expert_linear_bwd")
    return gx, gw, gb


def gs_expert_route_fwd(logits, topk, keep=None, renormalise=True, balance=True, workspace=None,
                        stream=None):
    """The choice of experts for logits (tokens, experts): (ids int32 (tokens,
    topk), weights float32 (tokens, topk), counts int32 (experts + 1,), loss
    float32 (1,)), the last two None without balance.  keep bool (tokens,):
    the tokens that take part (None: all); the others' ids are -1.  counts'
    last element is how many tokens take part."""
    dt = _dtype(logits, "logits")
    if logits.dim() != 2:
        _refuse("logits: (tokens, experts) expected")
    T, E = logits.shape
    lp, ldl = _rows(logits, "logits")
    if keep is not None and (keep.dtype not in (torch.bool, torch.uint8) or keep.shape != (T,)):
        _refuse("keep: bool (tokens,) expected")
    if not 0 < topk <= E:
        _refuse("topk: at least one choice and at most every expert expected")
    ids = _new((T, topk), torch.int32, logits, stream)
    weights = _new((T, topk), torch.float32, logits, stream)
    counts = loss = ws = None
    n_bytes = 0
    L = lib()
    if balance:
        counts = _new((E + 1,), torch.int32, logits, stream)
        loss = _new((1,), torch.float32, logits, stream)
        n_bytes = L.gs_expert_route_workspace_size(T, E)
        ws = _workspace(workspace, n_bytes, logits, stream) if n_bytes else None
    _check(L.gs_expert_route_fwd(lp, ldl, _ptr(keep), T, topk, E, dt, int(renormalise), _ptr(ids),
                                 _ptr(weights), _ptr(counts), _ptr(loss), _ptr(ws), n_bytes,
                                 _on(stream, logits, keep, ws)), "gs_expert_route_fwd")
    return ids, weights, counts, loss


def gs_expert_route_bwd(logits, ids, counts=None, grad_weights=None, grad_loss=None,
                        renormalise=True, d_status=None, out=None, stream=None):
    """The gradient in the logits of gs_expert_route_fwd's weights
    (grad_weights float32 (tokens, topk)) and loss (grad_loss, one float32 on
    the device), each None for zeros; counts are needed with grad_loss."""
    dt = _dtype(logits, "logits")
    if logits.dim() != 2 or ids.dim() != 2 or ids.dtype != torch.int32 or \
            ids.shape[0] != logits.shape[0]:
        _refuse("logits (tokens, experts) and ids int32 (tokens, topk) expected")
    T, E = logits.shape
    k = ids.shape[1]
    lp, ldl = _rows(logits, "logits")
    if grad_weights is not None:
        _same(grad_weights, ids.shape, torch.float32, "grad_weights")
    if grad_loss is not None:
        if grad_loss.numel() != 1 or grad_loss.dtype != torch.float32:
            _refuse("grad_loss: one float32 expected")
        if counts is None:
            _refuse("counts: needed with grad_loss")
        _same(counts, (E + 1,), torch.int32, "counts")
    if out is None:
        grad = _new((T, E), logits.dtype, logits, stream)
        op, ldo = grad.data_ptr() or None, E
    else:
        grad = _same(out, (T, E), logits.dtype, "out")
        op, ldo = _rows(grad, "out")
    _check(lib().gs_expert_route_bwd(lp, ldl, _ptr(ids), _ptr(counts), _ptr(grad_weights),
                                     _ptr(grad_loss), T, k, E, dt, int(renormalise), op, ldo,
                                     _ptr(d_status),
                                     _on(stream, logits, ids, counts, grad_weights, grad_loss,
                                         d_status, out)),
           "gs_expert_route_bwd")
    return grad


# 8-bit rows: q float8_e4m3fn (..., channels rounded up to 16) and scales
# float8_e8m0fnu (..., a power of two for every 128 channels, rounded up to 4).
_Q8, _S8 = torch.float8_e4m3fn, torch.float8_e8m0fnu


def _widths8(channels):
    return (channels + 15) // 16 * 16, (channels + 511) // 512 * 4


def _rows8(q, scales, channels, what):
    """(pointer to q, pointer to scales) of 8-bit rows of `channels`."""
    wide, blocks = _widths8(channels)
    shape = q.shape
    if q.dtype is not _Q8 or scales.dtype is not _S8 or not shape or shape[-1] != wide or \
            scales.shape != shape[:-1] + (blocks,):
        _refuse(f"{what}: float8_e4m3fn (..., {wide}) and float8_e8m0fnu (..., {blocks}) expected")
    return _ptr(q), _ptr(scales)


def gs_rows_pack8(x, stream=None):
    """The rows of x (..., channels) in 8 bits: (q float8_e4m3fn (..., channels
    rounded up to 16), scales float8_e8m0fnu (..., one for every 128 channels,
    rounded up to 4)); zeros behind the last channel and block."""
    dt = _dtype(x, "x")
    xp, ldx = _rows(x, "x")
    ch = x.shape[-1]
    wide, blocks = _widths8(ch)
    q = _new((*x.shape[:-1], wide), _Q8, x, stream)
    scales = _new((*x.shape[:-1], blocks), _S8, x, stream)
    _check(lib().gs_rows_pack8(xp, ldx, x.numel() // ch if ch else 0, ch, dt, _ptr(q),
                               _ptr(scales), _on(stream, x)), "gs_rows_pack8")
    return q, scales


def gs_rows_unpack8(q, scales, channels, dtype=torch.bfloat16, out=None, stream=None):
    """The values (..., channels) of gs_rows_pack8's rows, rounded to dtype."""
    qp, sp = _rows8(q, scales, channels, "q, scales")
    shape = (*q.shape[:-1], channels)
    if out is None:
        y = _new(shape, dtype, q, stream)
        yp, ldy = y.data_ptr() or None, channels
    else:
        y = _same(out, shape, dtype, "out")
        yp, ldy = _rows(y, "out")
    _check(lib().gs_rows_unpack8(qp, sp, q.numel() // q.shape[-1] if channels else 0, channels,
                                 _dtype(y, "dtype"), yp, ldy, _on(stream, q, scales, out)),
           "gs_rows_unpack8")
    return y


def _linear8_shapes(xs, offsets, weight, channels):
    E = _experts(offsets)
    w, x = weight.shape, xs.shape
    if len(w) != 3 or w[0] != E or len(x) != 2 or channels < 1:
        _refuse("xs (rows, ...) and weight (experts, out_features, ...) expected")
    return x[0], E, w[1]


def gs_expert_linear8_fwd(xs, xs_scales, offsets, weight, weight_scales, in_features, bias=None,
                          dtype=torch.bfloat16, d_status=None, out=None, stream=None):
    """gs_expert_linear_fwd of 8-bit rows (gs_rows_pack8): xs (rows, ...),
    weight (experts, out_features, ...) of in_features channels, bias
    (experts, out_features) of dtype or None.  Returns ys (rows,
    out_features) of dtype."""
    R, E, o = _linear8_shapes(xs, offsets, weight, in_features)
    xp, xsp = _rows8(xs, xs_scales, in_features, "xs")
    wp, wsp = _rows8(weight, weight_scales, in_features, "weight")
    if bias is not None:
        _same(bias, (E, o), dtype, "bias")
    ys = _new((R, o), dtype, xs, stream) if out is None else _same(out, (R, o), dtype, "out")
    _check(lib().gs_expert_linear8_fwd(xp, xsp, _ptr(offsets), wp, wsp, _ptr(bias), R, E,
                                       in_features, o, _dtype(ys, "dtype"), _ptr(ys),
                                       _ptr(d_status),
                                       _on(stream, xs, xs_scales, offsets, weight, weight_scales,
                                           bias, d_status, out)), "gs_expert_linear8_fwd")
    return ys


def gs_expert_linear8_bwd(grad_ys, xs, xs_scales, offsets, weight, weight_scales, in_features,
                          bias=True, input=True, d_status=None, workspace=None, stream=None):
    """Gradients of gs_expert_linear8_fwd in the values of its 8-bit rows:
    (grad_xs, grad_weight, grad_bias) of grad_ys' type, the first None without
    `input`, the last None without `bias`."""
    dt = _dtype(grad_ys, "grad_ys")
    R, E, o = _linear8_shapes(xs, offsets, weight, in_features)
    xp, xsp = _rows8(xs, xs_scales, in_features, "xs")
    wp, wsp = _rows8(weight, weight_scales, in_features, "weight")
    _same(grad_ys, (R, o), grad_ys.dtype, "grad_ys")
    t = grad_ys.dtype
    gx = _new((R, in_features), t, grad_ys, stream) if input else None
    gw = _new((E, o, in_features), t, grad_ys, stream)
    gb = _new((E, o), t, grad_ys, stream) if bias else None
    L = lib()
    n_bytes = L.gs_expert_linear8_bwd_workspace_size(R, E, in_features, o, dt,
                                                     grad_ys.data_ptr() % 16 == 0)
    ws = _workspace(workspace, n_bytes, grad_ys, stream) if n_bytes else None
    _check(L.gs_expert_linear8_bwd(_ptr(grad_ys), xp, xsp, _ptr(offsets), wp, wsp, R, E,
                                   in_features, o, dt, _ptr(gx), _ptr(gw), _ptr(gb), _ptr(ws),
                                   n_bytes, _ptr(d_status),
                                   _on(stream, grad_ys, xs, xs_scales, offsets, weight,
                                       weight_scales, d_status, ws)),
           "gs_expert_linear8_bwd")
    return gx, gw, gb
