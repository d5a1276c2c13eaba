"""Python binding of libsga.so: vocab-sharded greedy token selection on GB300.

Argument marshalling only.  Each function has the name of the C entry point
it calls (declared in include/sga.h), takes torch CUDA tensors where the C
call takes device pointers, passes data_ptr() values and the current torch
stream, and raises SgaError on a non-zero status.  Every step of the path
runs in the library's CUDA kernels; there is no fallback: if libsga.so has
not been built, every call raises.

Stats tensors are int32 [rows, 2] (8 bytes per row: fp32 value bits, int32
id); ``stat_values``/``stat_ids`` view the two columns.

Method: vLLM PR #34049 (Solution: local argmax per vocab shard, gather of
(max_value, global_index), cross-rank reduce), PR #39419 (draft-to-target
map after the local argmax), PR #62604 (Purpose items 1-2: dim-0 gathered
per-shard stats, one verify kernel; fused get_top_tokens with padding mask
and torch.argmax order).
"""
import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_build", "libsga.so")

SGA_F32, SGA_BF16 = 0, 1
SGA_MAX_K = 15
SGA_MAX_VOCAB = 1 << 24
SGA_MAX_TOP = 32
SGA_MAX_TEACHER = 128
SGA_ACT_NONE, SGA_ACT_RELU, SGA_ACT_SILU, SGA_ACT_GELU, SGA_ACT_GELU_TANH = 0, 1, 2, 3, 4
SGA_DEVERR_K_RANGE, SGA_DEVERR_D2T_RANGE, SGA_DEVERR_TIMEOUT, SGA_DEVERR_LAYOUT = 1, 2, 4, 8

_lib = None


class SgaError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn} failed: {status} ({sga_status_string(status)})")


def lib():
    """The loaded libsga.so (ctypes), with argument types set."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with "
                "`python -m greedy_spec_decode_gb300.build` (or __graft_entry__.build())")
        L = ctypes.CDLL(LIB_PATH)
        i64, i32, vp, sz = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t
        sig = {
            "sga_version": ([], i32),
            "sga_status_string": ([i32], ctypes.c_char_p),
            "sga_local_argmax": ([vp, i32, i64, i64, i64, i64, i64, vp, vp], i32),
            "sga_local_argmax_shards": ([vp, i32, i64, i64, i32, vp, vp, i64, vp, vp], i32),
            "sga_block_slots": ([i64, i64, i64, i64], i64),
            "sga_local_argmax_blocks": ([vp, i32, i64, i64, i64, i64, i64, i64, i64, i32, vp,
                                         vp, vp], i32),
            "sga_local_argmax_blocks_shards": ([vp, i32, i64, i64, i32, vp, vp, i64, i64, i64,
                                                i32, vp, vp, vp], i32),
            "sga_shard_reduce": ([vp, i32, i64, vp, vp, vp, i64, vp], i32),
            "sga_greedy_verify": ([vp, i32, i32, vp, vp, i32, vp, vp, vp, vp, vp, vp], i32),
            "sga_greedy_verify_prefill": ([vp, i32, i32, vp, vp, vp, i32, vp, vp, vp, vp, vp,
                                           vp], i32),
            "sga_lmhead_argmax_workspace": ([i64, i64], sz),
            "sga_lmhead_argmax_shards_workspace": ([i64, i32, vp], sz),
            "sga_lmhead_argmax_shards": ([vp, i64, i64, vp, i32, vp, vp, i64, vp, vp, sz, vp], i32),
            "sga_lmhead_argmax_shards_fp8": ([vp, vp, i64, i64, vp, ctypes.c_float, i32, vp, vp,
                                              i64, vp, vp, sz, vp], i32),
            "sga_lmhead_argmax": ([vp, i64, i64, vp, i64, i64, i64, vp, vp, sz, vp], i32),
            "sga_lmhead_argmax_fp8": ([vp, vp, i64, i64, vp, ctypes.c_float, i64, i64, i64, vp,
                                       vp, sz, vp], i32),
            "sga_linear": ([vp, i64, i64, i64, vp, i64, i64, vp, i32, i32, vp, i64, vp, i64, vp,
                            i64, vp], i32),
            "sga_linear_grad_workspace": ([i64, i64, i64], sz),
            "sga_linear_grad": ([vp, i64, i64, i64, vp, i64, i32, vp, i64, i64, vp, i64, vp, i64,
                                 vp, i64, vp, i32, vp, sz, vp], i32),
            "sga_token_logprobs": ([vp, i32, i64, i64, i64, i64, vp, i32, vp, vp, vp, vp, vp,
                                    vp], i32),
            "sga_local_logprobs": ([vp, i32, i64, i64, i64, i64, i64, vp, i32, vp, vp, vp], i32),
            "sga_logprob_reduce": ([vp, vp, i32, i64, i32, vp, vp, vp, vp, vp, vp, vp], i32),
            "sga_token_logprobs_grad": ([vp, i32, i64, i64, i64, i64, i64, vp, vp, vp, vp, vp,
                                         i32, vp, vp, vp, i64, vp], i32),
            "sga_probs": ([vp, i32, i64, i64, i64, i64, vp, vp, i64, vp], i32),
            "sga_sampled_verify": ([vp, i64, i64, vp, i64, i64, i32, vp, vp, vp, vp, vp, i32, vp,
                                    vp, vp, vp, vp], i32),
            "sga_distill": ([vp, i32, i64, i64, i64, i64, vp, vp, i32, vp, ctypes.c_float, vp,
                             vp, vp, vp, vp, i64, vp], i32),
            "sga_distill_grad": ([vp, i32, i64, i64, i64, i64, vp, vp, i32, vp, ctypes.c_float,
                                  vp, vp, vp, vp, i64, vp], i32),
            "sga_device_error": ([ctypes.POINTER(ctypes.c_uint32)], i32),
            "sga_clear_device_error": ([], i32),
            "sga_selftest_wait_timeout": ([ctypes.c_uint64, vp, vp], i32),
        }
        for name, (args, res) in sig.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        _lib = L
    return _lib


def sga_version():
    return lib().sga_version()


def sga_status_string(status):
    return lib().sga_status_string(int(status)).decode()


def _check(fn, status):
    if status != 0:
        raise SgaError(fn, status)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _dtype_code(t):
    if t.dtype == torch.float32:
        return SGA_F32
    if t.dtype == torch.bfloat16:
        return SGA_BF16
    raise TypeError(f"logits must be float32 or bfloat16, got {t.dtype}")


def new_stats(rows, device="cuda"):
    """An int32 [rows, 2] tensor that holds `rows` stats."""
    return torch.empty((rows, 2), dtype=torch.int32, device=device)


def stat_values(stats):
    return stats[..., 0].view(torch.float32)


def stat_ids(stats):
    return stats[..., 1]


def sga_local_argmax(logits, shard_start, shard_width, org_vocab, out_stats, stream=None):
    """Per-shard argmax.  `logits` is a 2-D CUDA tensor whose column 0 is the
    shard's first id (a column slice of the full matrix, or a per-rank
    buffer), unit stride along the vocab; out_stats receives one stat per row
    (pass a slice of the gathered buffer to emulate all_gather on dim 0)."""
    if logits.dim() != 2 or (logits.size(1) > 1 and logits.stride(1) != 1):
        raise ValueError("logits must be 2-D with unit stride along the vocab")
    rows = logits.size(0)
    ld = logits.stride(0) if rows > 1 else max(logits.stride(0), shard_width)
    _check("sga_local_argmax", lib().sga_local_argmax(
        _ptr(logits), _dtype_code(logits), rows, ld, int(shard_start), int(shard_width),
        int(org_vocab), _ptr(out_stats), _stream(stream)))
    return out_stats


def sga_local_argmax_shards(logits, shards, org_vocab, out_stats, stream=None):
    """Per-shard argmax of several shards in one launch.  `logits` is a 2-D
    CUDA tensor whose column 0 is global id shards[0][0] (unit stride along
    the vocab); shards = [(start, width), ...] ascending; out_stats receives
    len(shards) * rows stats in shard-major (all_gather dim 0) order."""
    if logits.dim() != 2 or (logits.size(1) > 1 and logits.stride(1) != 1):
        raise ValueError("logits must be 2-D with unit stride along the vocab")
    n = len(shards)
    starts = (ctypes.c_int64 * n)(*[int(o) for o, _ in shards])
    widths = (ctypes.c_int64 * n)(*[int(w) for _, w in shards])
    rows = logits.size(0)
    ld = logits.stride(0) if rows > 1 else max(logits.stride(0), logits.size(1))
    _check("sga_local_argmax_shards", lib().sga_local_argmax_shards(
        _ptr(logits), _dtype_code(logits), rows, ld, n, starts, widths, int(org_vocab),
        _ptr(out_stats), _stream(stream)))
    return out_stats


def sga_block_slots(shard_start, shard_width, draft_block, bonus_block=None):
    """Stats per row that sga_local_argmax_blocks writes for one shard."""
    bonus_block = draft_block if bonus_block is None else bonus_block
    n = int(lib().sga_block_slots(int(shard_start), int(shard_width), int(draft_block),
                                  int(bonus_block)))
    _check("sga_block_slots", n if n < 0 else 0)
    return n


def sga_local_argmax_blocks(logits, shard_start, shard_width, org_vocab, draft_block,
                            out_stats, bonus_block=None, cu_num_draft=None, stream=None):
    """Block-granular stats of one shard: for every row, the argmax of each
    fixed global block of ids meeting the shard.  `logits` as for
    sga_local_argmax; out_stats receives sga_block_slots(...) * rows stats,
    piece-major.  With cu_num_draft (int32 CUDA tensor [N + 1]) the bonus row
    of each request uses bonus_block."""
    if logits.dim() != 2 or (logits.size(1) > 1 and logits.stride(1) != 1):
        raise ValueError("logits must be 2-D with unit stride along the vocab")
    bonus_block = draft_block if bonus_block is None else bonus_block
    rows = logits.size(0)
    ld = logits.stride(0) if rows > 1 else max(logits.stride(0), shard_width)
    num_reqs = 0 if cu_num_draft is None else cu_num_draft.numel() - 1
    _check("sga_local_argmax_blocks", lib().sga_local_argmax_blocks(
        _ptr(logits), _dtype_code(logits), rows, ld, int(shard_start), int(shard_width),
        int(org_vocab), int(draft_block), int(bonus_block), int(num_reqs), _ptr(cu_num_draft),
        _ptr(out_stats), _stream(stream)))
    return out_stats


def sga_local_argmax_blocks_shards(logits, shards, org_vocab, draft_block, out_stats,
                                   bonus_block=None, cu_num_draft=None, stream=None):
    """Block-granular stats of several shards in one launch.  `logits` is a
    2-D CUDA tensor whose column 0 is global id shards[0][0]; shards =
    [(start, width), ...] ascending; out_stats receives the shards' slots
    concatenated in shard order (see sga_block_slots), piece-major."""
    if logits.dim() != 2 or (logits.size(1) > 1 and logits.stride(1) != 1):
        raise ValueError("logits must be 2-D with unit stride along the vocab")
    bonus_block = draft_block if bonus_block is None else bonus_block
    n = len(shards)
    starts = (ctypes.c_int64 * n)(*[int(o) for o, _ in shards])
    widths = (ctypes.c_int64 * n)(*[int(w) for _, w in shards])
    rows = logits.size(0)
    ld = logits.stride(0) if rows > 1 else max(logits.stride(0), logits.size(1))
    num_reqs = 0 if cu_num_draft is None else cu_num_draft.numel() - 1
    _check("sga_local_argmax_blocks_shards", lib().sga_local_argmax_blocks_shards(
        _ptr(logits), _dtype_code(logits), rows, ld, n, starts, widths, int(org_vocab),
        int(draft_block), int(bonus_block), int(num_reqs), _ptr(cu_num_draft),
        _ptr(out_stats), _stream(stream)))
    return out_stats


def sga_shard_reduce(stats, num_shards, rows, out_ids, out_vals=None, d2t=None, stream=None):
    """Global argmax per row from the gathered stats [num_shards * rows];
    with d2t (int64 CUDA tensor) the ids are mapped k -> k + d2t[k]."""
    _check("sga_shard_reduce", lib().sga_shard_reduce(
        _ptr(stats), int(num_shards), int(rows), _ptr(out_vals), _ptr(out_ids), _ptr(d2t),
        0 if d2t is None else d2t.numel(), _stream(stream)))
    return out_ids


def sga_greedy_verify(stats, num_shards, cu_num_draft, draft_tokens, max_k, out_sampled,
                      out_num_sampled, out_num_rejected, out_bonus, out_target_ids=None,
                      stream=None):
    """Fused cross-shard reduce + greedy verification (see include/sga.h)."""
    num_reqs = cu_num_draft.numel() - 1
    _check("sga_greedy_verify", lib().sga_greedy_verify(
        _ptr(stats), int(num_shards), int(num_reqs), _ptr(cu_num_draft),
        _ptr(draft_tokens) if draft_tokens is not None and draft_tokens.numel() else None,
        int(max_k), _ptr(out_sampled), _ptr(out_num_sampled), _ptr(out_num_rejected),
        _ptr(out_bonus), _ptr(out_target_ids), _stream(stream)))


def sga_greedy_verify_prefill(stats, num_shards, cu_num_draft, draft_tokens, in_prefill, max_k,
                              out_sampled, out_num_sampled, out_num_rejected, out_bonus,
                              out_target_ids=None, stream=None):
    """sga_greedy_verify where in_prefill (a uint8/bool CUDA tensor [num_reqs],
    or None) marks the requests still in prefill, which emit nothing."""
    num_reqs = cu_num_draft.numel() - 1
    if in_prefill is not None and in_prefill.dtype not in (torch.uint8, torch.bool):
        raise ValueError("in_prefill must be a uint8 or bool tensor")
    _check("sga_greedy_verify_prefill", lib().sga_greedy_verify_prefill(
        _ptr(stats), int(num_shards), int(num_reqs), _ptr(cu_num_draft),
        _ptr(draft_tokens) if draft_tokens is not None and draft_tokens.numel() else None,
        _ptr(in_prefill), int(max_k), _ptr(out_sampled), _ptr(out_num_sampled),
        _ptr(out_num_rejected), _ptr(out_bonus), _ptr(out_target_ids), _stream(stream)))


def sga_lmhead_argmax_workspace(M, shard_width):
    return int(lib().sga_lmhead_argmax_workspace(int(M), int(shard_width)))


def sga_lmhead_argmax(hidden, weight_shard, shard_start, org_vocab, out_stats, workspace,
                      stream=None):
    """Fused LM-head GEMM + per-shard argmax.  hidden: bf16 [M, H] contiguous;
    weight_shard: bf16 [shard_width, H] contiguous; workspace: a CUDA tensor of
    at least sga_lmhead_argmax_workspace(M, shard_width) bytes."""
    if not (hidden.is_contiguous() and weight_shard.is_contiguous()):
        raise ValueError("hidden and weight_shard must be contiguous")
    M, H = hidden.shape
    width = weight_shard.size(0)
    if weight_shard.size(1) != H:
        raise ValueError("hidden and weight_shard must share H")
    nbytes = workspace.numel() * workspace.element_size()
    _check("sga_lmhead_argmax", lib().sga_lmhead_argmax(
        _ptr(hidden), M, H, _ptr(weight_shard), int(shard_start), width, int(org_vocab),
        _ptr(out_stats), _ptr(workspace), nbytes, _stream(stream)))
    return out_stats


def sga_lmhead_argmax_fp8(hidden_q, hidden_scale, weight_q, weight_scale, shard_start,
                          org_vocab, out_stats, workspace, stream=None):
    """Fused fp8 (E4M3) LM-head GEMM + per-shard argmax.  hidden_q: uint8 [M, H]
    codes, hidden_scale: float32 [M] CUDA tensor or None, weight_q: uint8
    [shard_width, H] codes, weight_scale: positive float (see include/sga.h)."""
    if not (hidden_q.is_contiguous() and weight_q.is_contiguous()):
        raise ValueError("hidden_q and weight_q must be contiguous")
    if hidden_q.dtype != torch.uint8 or weight_q.dtype != torch.uint8:
        raise TypeError("fp8 operands are passed as uint8 E4M3 codes")
    M, H = hidden_q.shape
    width = weight_q.size(0)
    if weight_q.size(1) != H:
        raise ValueError("hidden_q and weight_q must share H")
    nbytes = workspace.numel() * workspace.element_size()
    _check("sga_lmhead_argmax_fp8", lib().sga_lmhead_argmax_fp8(
        _ptr(hidden_q), _ptr(hidden_scale), M, H, _ptr(weight_q), float(weight_scale),
        int(shard_start), width, int(org_vocab), _ptr(out_stats), _ptr(workspace), nbytes,
        _stream(stream)))
    return out_stats


def _shard_arrays(shards):
    n = len(shards)
    return (n, (ctypes.c_int64 * n)(*[int(o) for o, _ in shards]),
            (ctypes.c_int64 * n)(*[int(w) for _, w in shards]))


def sga_lmhead_argmax_shards_workspace(M, shards):
    n, _, widths = _shard_arrays(shards)
    return int(lib().sga_lmhead_argmax_shards_workspace(int(M), n, widths))


def sga_lmhead_argmax_shards(hidden, weight, shards, org_vocab, out_stats, workspace,
                             stream=None):
    """Fused LM head + argmax of several shards of one weight buffer in one call:
    weight: bf16 [rows, H] contiguous, row 0 = global id shards[0][0]; shards =
    [(start, width), ...] ascending; out_stats receives len(shards) * M stats,
    shard-major."""
    if not (hidden.is_contiguous() and weight.is_contiguous()):
        raise ValueError("hidden and weight must be contiguous")
    M, H = hidden.shape
    if weight.size(1) != H:
        raise ValueError("hidden and weight must share H")
    n, starts, widths = _shard_arrays(shards)
    if starts[n - 1] - starts[0] + widths[n - 1] > weight.size(0):
        raise ValueError("weight does not span the shards")
    nbytes = workspace.numel() * workspace.element_size()
    _check("sga_lmhead_argmax_shards", lib().sga_lmhead_argmax_shards(
        _ptr(hidden), M, H, _ptr(weight), n, starts, widths, int(org_vocab), _ptr(out_stats),
        _ptr(workspace), nbytes, _stream(stream)))
    return out_stats


def sga_lmhead_argmax_shards_fp8(hidden_q, hidden_scale, weight_q, weight_scale, shards,
                                 org_vocab, out_stats, workspace, stream=None):
    """sga_lmhead_argmax_shards with E4M3 operands (uint8 codes) and one weight
    scale for the whole weight buffer (see include/sga.h)."""
    if not (hidden_q.is_contiguous() and weight_q.is_contiguous()):
        raise ValueError("hidden_q and weight_q must be contiguous")
    if hidden_q.dtype != torch.uint8 or weight_q.dtype != torch.uint8:
        raise TypeError("fp8 operands are passed as uint8 E4M3 codes")
    M, H = hidden_q.shape
    if weight_q.size(1) != H:
        raise ValueError("hidden_q and weight_q must share H")
    n, starts, widths = _shard_arrays(shards)
    if starts[n - 1] - starts[0] + widths[n - 1] > weight_q.size(0):
        raise ValueError("weight_q does not span the shards")
    nbytes = workspace.numel() * workspace.element_size()
    _check("sga_lmhead_argmax_shards_fp8", lib().sga_lmhead_argmax_shards_fp8(
        _ptr(hidden_q), _ptr(hidden_scale), M, H, _ptr(weight_q), float(weight_scale), n,
        starts, widths, int(org_vocab), _ptr(out_stats), _ptr(workspace), nbytes,
        _stream(stream)))
    return out_stats


def _bf16_rows(t, shape, name):
    """(address, row stride) of a bf16 tensor of that shape with unit column
    stride; (None, 0) for None."""
    if t is None:
        return None, 0
    if t.dtype is not _BF16 or t.shape != shape:
        raise ValueError(f"{name} must be bf16 {list(shape)}")
    row, col = t.stride()
    rows, cols = shape
    if col != 1 and cols > 1:
        raise ValueError(f"{name} must have unit column stride")
    return t.data_ptr(), row if rows > 1 else cols  # a single row's stride is never used


def _bias(t, n, name):
    """(address, dtype code) of a float32 or bf16 vector of n, or (None, SGA_F32)."""
    if t is None:
        return None, SGA_F32
    dtype = t.dtype
    if (dtype is not _F32 and dtype is not _BF16) or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 or bf16 tensor of {n} elements")
    return t.data_ptr(), SGA_F32 if dtype is _F32 else SGA_BF16


def sga_linear(x, weight, out, bias=None, act=SGA_ACT_NONE, residual=None, out_preact=None,
               stream=None):
    """out = act(x . weight^T + bias) + residual.  x: bf16 [M, K], weight: bf16
    [N, K], out / residual / out_preact: bf16 [M, N] (unit column stride, any
    row stride; x and weight rows 16-byte aligned), bias: float32 or bf16 [N].
    out may be residual itself; out_preact receives x . weight^T + bias, which
    sga_linear_grad needs when there is an activation (see include/sga.h)."""
    M, K = shape_x = x.shape
    N = weight.size(0)
    shape_y = (M, N)
    px, ldx = _bf16_rows(x, shape_x, "x")
    pw, ldw = _bf16_rows(weight, (N, K), "weight")
    po, ldo = _bf16_rows(out, shape_y, "out")
    pr, ldr = _bf16_rows(residual, shape_y, "residual")
    pp, ldp = _bf16_rows(out_preact, shape_y, "out_preact")
    pb, code = _bias(bias, N, "bias")
    _on_gpu(x, weight, out, bias, residual, out_preact)
    _check("sga_linear", lib().sga_linear(
        px, M, K, ldx, pw, N, ldw, pb, code, int(act), pr, ldr, pp, ldp, po, ldo,
        _raw_stream(stream)))
    return out


def sga_linear_grad_workspace(M, N, K):
    return int(lib().sga_linear_grad_workspace(int(M), int(N), int(K)))


def sga_linear_grad(grad_out, x, weight, workspace, act=SGA_ACT_NONE, preact=None, grad_x=None,
                    grad_weight=None, grad_bias=None, stream=None):
    """Gradient of sga_linear with respect to x, weight and bias (each output
    bf16 like its operand, grad_bias float32 or bf16, or None); the residual's
    gradient is grad_out itself.  preact: sga_linear's out_preact; workspace: a
    CUDA tensor of at least sga_linear_grad_workspace(M, N, K) bytes."""
    M, K = shape_x = x.shape
    N = weight.size(0)
    shape_w, shape_y = (N, K), (M, N)
    px, ldx = _bf16_rows(x, shape_x, "x")
    pw, ldw = _bf16_rows(weight, shape_w, "weight")
    pg, ldg = _bf16_rows(grad_out, shape_y, "grad_out")
    pp, ldp = _bf16_rows(preact, shape_y, "preact")
    pgx, ldgx = _bf16_rows(grad_x, shape_x, "grad_x")
    pgw, ldgw = _bf16_rows(grad_weight, shape_w, "grad_weight")
    pb, code = _bias(grad_bias, N, "grad_bias")
    _on_gpu(grad_out, x, weight, workspace, preact, grad_x, grad_weight, grad_bias)
    _check("sga_linear_grad", lib().sga_linear_grad(
        pg, M, N, ldg, pp, ldp, int(act), px, K, ldx, pw, ldw, pgx, ldgx, pgw, ldgw, pb, code,
        workspace.data_ptr(), workspace.numel() * workspace.element_size(), _raw_stream(stream)))


# The calls above and below run beside single-token steps of a few microseconds, so their
# marshalling is kept short: plain integers for pointers (ctypes takes them for
# c_void_p) and the raw handle of the current stream.


_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32
# (absent from builds of torch without CUDA; only reached with CUDA tensors)
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)


def _raw_stream(stream):
    if stream is None:
        return _current_raw_stream(_current_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check_out(t, dtype, numel, name):
    """Address of a contiguous tensor of `dtype` with `numel` elements, or None."""
    if t is None:
        return None
    if t.dtype is not dtype or t.numel() != numel or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {numel} elements")
    return t.data_ptr()


def _on_gpu(*tensors):
    """Tensors of the current device, on whose stream the calls run."""
    here = None
    for t in tensors:
        if t is None:
            continue
        at = t.get_device()      # -1: host memory
        if at != here:
            if at < 0:
                raise ValueError("CUDA tensors are needed")
            if here is not None or at != _current_device():
                raise ValueError("CUDA tensors of the current device are needed")
            here = at


def _logits_2d(logits):
    shape = logits.shape
    if len(shape) != 2:
        raise ValueError("logits must be 2-D")
    rows, width = shape
    ld, col = logits.stride()
    if col != 1 and width > 1:
        raise ValueError("logits must have unit stride along the vocab")
    return rows, width, ld if rows > 1 else max(ld, width), _dtype_code(logits)


def _row_outputs(rows, tokens, out_logprob, out_entropy, out_lse, out_top_ids, out_top_logprobs):
    """top_k and the addresses of the per-row tensors of the log-probability calls."""
    top = out_top_ids if out_top_ids is not None else out_top_logprobs
    k = 0 if top is None else top.size(-1)
    f32, i32 = _F32, _I32
    return k, (_check_out(tokens, i32, rows, "tokens"),
               _check_out(out_logprob, f32, rows, "out_logprob"),
               _check_out(out_entropy, f32, rows, "out_entropy"),
               _check_out(out_lse, f32, rows, "out_lse"),
               _check_out(out_top_ids, i32, rows * k, "out_top_ids"),
               _check_out(out_top_logprobs, f32, rows * k, "out_top_logprobs"))


def sga_token_logprobs(logits, org_vocab, tokens=None, out_logprob=None, out_entropy=None,
                       out_lse=None, out_top_ids=None, out_top_logprobs=None, stream=None):
    """Log probability of each row's token (int32 [rows]) over a whole
    vocabulary, with the row's entropy, log-sum-exp and the top_k best ids with
    their log probabilities.  logits: 2-D, unit stride along the vocab; outputs
    are contiguous CUDA tensors or None: float32 [rows], and int32 / float32
    [rows, top_k], whose last size is top_k (see include/sga.h)."""
    rows, width, ld, code = _logits_2d(logits)
    k, (tok, *outs) = _row_outputs(rows, tokens, out_logprob, out_entropy, out_lse, out_top_ids,
                                   out_top_logprobs)
    _on_gpu(logits, tokens, out_logprob, out_entropy, out_lse, out_top_ids, out_top_logprobs)
    _check("sga_token_logprobs", lib().sga_token_logprobs(
        logits.data_ptr(), code, rows, ld, width, int(org_vocab), tok, k, *outs,
        _raw_stream(stream)))


def sga_local_logprobs(logits, shard_start, shard_width, org_vocab, tokens, out_parts,
                       out_top=None, stream=None):
    """One vocab shard's part of sga_token_logprobs.  logits: 2-D, column 0 =
    global id shard_start; out_parts: float32 [rows, 4]; out_top: int32 [rows,
    top_k, 2] stats, or None (pass slices of the gathered buffers to emulate
    all_gather on dim 0)."""
    rows, width, ld, code = _logits_2d(logits)
    if width < shard_width:
        raise ValueError("logits has fewer columns than the shard")
    k = 0 if out_top is None else out_top.size(-2)
    _on_gpu(logits, tokens, out_parts, out_top)
    _check("sga_local_logprobs", lib().sga_local_logprobs(
        logits.data_ptr(), code, rows, ld, int(shard_start), int(shard_width),
        int(org_vocab), _check_out(tokens, _I32, rows, "tokens"), k,
        _check_out(out_parts, _F32, 4 * rows, "out_parts"),
        _check_out(out_top, _I32, 2 * k * rows, "out_top"), _raw_stream(stream)))
    return out_parts


def sga_logprob_reduce(parts, tops, num_shards, tokens=None, out_logprob=None, out_entropy=None,
                       out_lse=None, out_top_ids=None, out_top_logprobs=None, stream=None):
    """Results of sga_token_logprobs from the gathered parts (float32
    [num_shards, rows, 4]) and lists (int32 [num_shards, rows, top_k, 2] or
    None)."""
    num_shards = int(num_shards)
    if num_shards < 1:
        raise ValueError("num_shards must be at least 1")
    rows = parts.numel() // (4 * num_shards)
    k, (tok, *outs) = _row_outputs(rows, tokens, out_logprob, out_entropy, out_lse, out_top_ids,
                                   out_top_logprobs)
    if k and tops is None:
        raise ValueError("alternatives are asked for without tops")
    _on_gpu(parts, tops, tokens, out_logprob, out_entropy, out_lse, out_top_ids,
            out_top_logprobs)
    _check("sga_logprob_reduce", lib().sga_logprob_reduce(
        _check_out(parts, _F32, 4 * rows * num_shards, "parts"),
        _check_out(tops, _I32, 2 * k * rows * num_shards, "tops") if k else None,
        num_shards, rows, k, tok, *outs, _raw_stream(stream)))


def sga_token_logprobs_grad(logits, shard_start, org_vocab, tokens, lse, entropy, grad_logprob,
                            out_grad, grad_entropy=None, top_ids=None, grad_top=None,
                            stream=None):
    """Gradient of sga_token_logprobs' log probabilities, entropy and
    alternatives with respect to the logits (a whole vocabulary, shard_start 0,
    or one shard).  lse, entropy: the forward results; the upstream gradients
    are float32 or None; out_grad: like logits, or logits itself."""
    rows, width, ld, code = _logits_2d(logits)
    if out_grad.dtype != logits.dtype or out_grad.shape != logits.shape or (
            width > 1 and out_grad.stride(1) != 1):
        raise ValueError("out_grad must match logits, unit stride along the vocab")
    ldg = out_grad.stride(0) if rows > 1 else max(out_grad.stride(0), width)
    k = 0 if top_ids is None else top_ids.size(-1)
    f32, i32 = _F32, _I32
    _on_gpu(logits, tokens, lse, entropy, grad_logprob, grad_entropy, top_ids, grad_top,
            out_grad)
    _check("sga_token_logprobs_grad", lib().sga_token_logprobs_grad(
        logits.data_ptr(), code, rows, ld, int(shard_start), width, int(org_vocab),
        _check_out(tokens, i32, rows, "tokens"), _check_out(lse, f32, rows, "lse"),
        _check_out(entropy, f32, rows, "entropy"),
        _check_out(grad_logprob, f32, rows, "grad_logprob"),
        _check_out(grad_entropy, f32, rows, "grad_entropy"), k,
        _check_out(top_ids, i32, rows * k, "top_ids"),
        _check_out(grad_top, f32, rows * k, "grad_top"), out_grad.data_ptr(), ldg,
        _raw_stream(stream)))
    return out_grad


# The calls below take up to 13 tensors, so each is looked at once: its layout, and that
# it lies where the call's first one does, which _stream_on then finds to be the current
# device (looked at apart, as above, a call takes 0.5 us longer).


def _vec(t, dtype, numel, name, here):
    """Address of a contiguous tensor of `dtype` with `numel` elements on device
    `here`, or None."""
    if t is None:
        return None
    if t.dtype is not dtype or t.numel() != numel or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {numel} elements")
    if t.get_device() != here:
        raise ValueError(f"{name} must be on the device of the first tensor")
    return t.data_ptr()


def _probs_2d(t, name, here):
    """(rows, columns, row stride, address) of fp32 probabilities."""
    shape = t.shape
    if t.dtype is not _F32 or len(shape) != 2:
        raise ValueError(f"{name} must be a 2-D float32 tensor")
    rows, width = shape
    ld, col = t.stride()
    if col != 1 and width > 1:
        raise ValueError(f"{name} must have unit stride along the vocab")
    if t.get_device() != here:
        raise ValueError(f"{name} must be on the device of the first tensor")
    return rows, width, ld if rows > 1 else max(ld, width), t.data_ptr()


def _stream_on(here, stream):
    """The raw handle of `stream`, or of the current one of device `here`, which has to be
    the current device."""
    if here < 0:
        raise ValueError("CUDA tensors are needed")
    if here != _current_device():
        raise ValueError("CUDA tensors of the current device are needed")
    return _current_raw_stream(here) if stream is None else _raw_stream(stream)


def sga_probs(logits, org_vocab, out_probs, temperature=None, stream=None):
    """Probabilities of logits rows at a temperature (float32 [rows], 0 = one at
    the argmax; None = 1).  logits: 2-D, unit stride along the vocab; out_probs:
    float32 of the same shape, or float32 logits themselves; ids past org_vocab
    get 0 (see include/sga.h)."""
    rows, width, ld, code = _logits_2d(logits)
    here = logits.get_device()
    out_rows, out_width, ldp, out = _probs_2d(out_probs, "out_probs", here)
    if out_rows != rows or out_width != width:
        raise ValueError("out_probs must have the shape of logits")
    temps = _vec(temperature, _F32, rows, "temperature", here)
    _check("sga_probs", lib().sga_probs(
        logits.data_ptr(), code, rows, ld, width, int(org_vocab), temps, out, ldp,
        _stream_on(here, stream)))
    return out_probs


def sga_sampled_verify(target_probs, draft_probs, cu_num_draft, draft_tokens, accept_u, sample_u,
                       max_k, out_sampled, out_num_sampled, out_num_rejected, out_last,
                       in_prefill=None, stream=None):
    """Verification of drafted tokens by rejection sampling.  target_probs:
    float32 [D + num_reqs, vocab] (rows as sga_greedy_verify's), draft_probs:
    float32 [D, vocab], or None for drafts without probabilities; draft_tokens
    int32 [D], accept_u float32 [D], sample_u float32 [num_reqs] (uniform in
    [0, 1)); in_prefill: uint8 / bool [num_reqs] or None.  Outputs: int32
    [num_reqs, max_k + 1] and int32 [num_reqs] (see include/sga.h)."""
    here = target_probs.get_device()
    rows, vocab, ldt, target = _probs_2d(target_probs, "target_probs", here)
    n, max_k = cu_num_draft.numel() - 1, int(max_k)
    drafts = rows - n
    if n < 0 or drafts < 0:
        raise ValueError("target_probs must have a row per draft and one per request")
    ldd, draft = 0, None
    if draft_probs is not None:
        d_rows, d_width, ldd, draft = _probs_2d(draft_probs, "draft_probs", here)
        if d_rows != drafts or d_width != vocab:
            raise ValueError("draft_probs must have a row per draft, as wide as target_probs")
        if drafts == 0:
            draft = None
    prefill = None
    if in_prefill is not None:
        if in_prefill.dtype not in (torch.uint8, torch.bool):
            raise ValueError("in_prefill must be a uint8 or bool tensor")
        prefill = _vec(in_prefill, in_prefill.dtype, n, "in_prefill", here)
    f32, i32 = _F32, _I32
    _check("sga_sampled_verify", lib().sga_sampled_verify(
        target, rows, ldt, draft, ldd, vocab, n,
        _vec(cu_num_draft, i32, n + 1, "cu_num_draft", here),
        _vec(draft_tokens, i32, drafts, "draft_tokens", here), prefill,
        _vec(accept_u, f32, drafts, "accept_u", here), _vec(sample_u, f32, n, "sample_u", here),
        max_k, _vec(out_sampled, i32, n * (max_k + 1), "out_sampled", here),
        _vec(out_num_sampled, i32, n, "out_num_sampled", here),
        _vec(out_num_rejected, i32, n, "out_num_rejected", here),
        _vec(out_last, i32, n, "out_last", here), _stream_on(here, stream)))


def _distill(name, logits, org_vocab, teacher_ids, teacher_logits, teacher_lse, temperature,
             loss, lse, lse_rest, lse_names, grad_loss, out_grad, stream):
    """The two distillation calls, which differ in the sums that they give or take."""
    rows, width, ld, code = _logits_2d(logits)
    here = logits.get_device()
    f32 = _F32
    shape = teacher_ids.shape
    if not shape:
        raise ValueError("teacher_ids must have a row per row of logits")
    k = shape[-1]
    ids = _vec(teacher_ids, _I32, rows * k, "teacher_ids", here)
    if teacher_logits.dim() > 1 and teacher_logits.shape[-1] != k:  # (of the size, not the order)
        raise ValueError("teacher_logits must have teacher_ids' k entries per row")
    z = _vec(teacher_logits, f32, rows * k, "teacher_logits", here)
    t_lse = _vec(teacher_lse, f32, rows, "teacher_lse", here)
    lse = _vec(lse, f32, rows, lse_names[0], here)
    rest = _vec(lse_rest, f32, rows, lse_names[1], here)
    up = _vec(grad_loss, f32, rows, "grad_loss", here)
    grad, ldg = None, 0
    if out_grad is not None:
        if out_grad.dtype is not logits.dtype or out_grad.shape != (rows, width):
            raise ValueError("out_grad must match logits")
        ldg, col = out_grad.stride()
        if col != 1 and width > 1:
            raise ValueError("out_grad must have unit stride along the vocab")
        if out_grad.get_device() != here:
            raise ValueError("out_grad must be on the device of the first tensor")
        grad = out_grad.data_ptr()
        if rows == 1 and ldg < width:
            ldg = width
    x, org_vocab, temperature = logits.data_ptr(), int(org_vocab), float(temperature)
    if name == "sga_distill":
        loss = _vec(loss, f32, rows, "out_loss", here)
        _check(name, lib().sga_distill(x, code, rows, ld, width, org_vocab, ids, z, k, t_lse,
                                       temperature, loss, lse, rest, up, grad, ldg,
                                       _stream_on(here, stream)))
    else:
        _check(name, lib().sga_distill_grad(x, code, rows, ld, width, org_vocab, ids, z, k, t_lse,
                                            temperature, lse, rest, up, grad, ldg,
                                            _stream_on(here, stream)))


def sga_distill(logits, org_vocab, teacher_ids, teacher_logits, out_loss=None, teacher_lse=None,
                temperature=1.0, out_lse=None, out_lse_rest=None, grad_loss=None, out_grad=None,
                stream=None):
    """Divergence of each row of a draft model's logits from a teacher's top
    logits: teacher_ids int32 / teacher_logits float32 [rows, k] (-1: no entry),
    teacher_lse float32 [rows], or None for the list by itself.  out_loss,
    out_lse, out_lse_rest: float32 [rows] or None; out_grad: the gradient with
    respect to logits times grad_loss (float32 [rows] or None), like logits, or
    logits itself, or None (see include/sga.h)."""
    _distill("sga_distill", logits, org_vocab, teacher_ids, teacher_logits, teacher_lse,
             temperature, out_loss, out_lse, out_lse_rest, ("out_lse", "out_lse_rest"), grad_loss,
             out_grad, stream)


def sga_distill_grad(logits, org_vocab, teacher_ids, teacher_logits, lse, lse_rest, out_grad,
                     teacher_lse=None, temperature=1.0, grad_loss=None, stream=None):
    """Gradient of sga_distill from the lse and lse_rest (float32 [rows]) that
    it gave; lse_rest may be None without teacher_lse.  out_grad: like logits, or
    logits itself."""
    _distill("sga_distill_grad", logits, org_vocab, teacher_ids, teacher_logits, teacher_lse,
             temperature, None, lse, lse_rest, ("lse", "lse_rest"), grad_loss, out_grad, stream)
    return out_grad


def sga_device_error():
    """Synchronise the current device and return its error word."""
    w = ctypes.c_uint32(0)
    _check("sga_device_error", lib().sga_device_error(ctypes.byref(w)))
    return w.value


def sga_clear_device_error():
    _check("sga_clear_device_error", lib().sga_clear_device_error())


def sga_selftest_wait_timeout(limit_ns, waited_ns=None, stream=None):
    """Run the bounded-wait self-test kernel (see include/sga.h)."""
    _check("sga_selftest_wait_timeout", lib().sga_selftest_wait_timeout(
        int(limit_ns), _ptr(waited_ns), _stream(stream)))


def sga_lmhead_argmax_noalloc(hidden, weight_shard, shard_start, org_vocab, out_stats,
                              stream=None):
    """sga_lmhead_argmax without a workspace, for callers that cannot allocate
    device memory on their decode path (a server or plugin that owns a
    pre-sized memory pool, or a loop where cudaMalloc would synchronise the
    device).  Partial statistics go to a fixed 4 MiB scratch array inside the
    library, shared by every call on the device: calls that overlap on the
    GPU race.  Rejects sga_lmhead_argmax_workspace(M, width) > 4 MiB with
    SGA_ERR_WORKSPACE.
    The first call on a device resolves the scratch address for that device;
    make it before any stream capture."""
    fn = lib().sga_lmhead_argmax_noalloc
    i64, vp = ctypes.c_int64, ctypes.c_void_p
    fn.argtypes = [vp, i64, i64, vp, i64, i64, i64, vp, vp]
    fn.restype = ctypes.c_int
    if not (hidden.is_contiguous() and weight_shard.is_contiguous()):
        raise ValueError("hidden and weight_shard must be contiguous")
    M, H = hidden.shape
    if weight_shard.size(1) != H:
        raise ValueError("hidden and weight_shard must share H")
    _check("sga_lmhead_argmax_noalloc", fn(
        _ptr(hidden), M, H, _ptr(weight_shard), int(shard_start), weight_shard.size(0),
        int(org_vocab), _ptr(out_stats), _stream(stream)))
    return out_stats
