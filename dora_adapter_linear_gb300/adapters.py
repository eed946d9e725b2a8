"""The plan of a batch whose rows have different adapters."""
from __future__ import annotations

import torch

from . import _lib as L


class AdapterPlan:
    """Rows by adapter and adapters by tile of one batch, on the device.  `update` refills it in place for
    a batch of as many rows, as a captured graph needs it; calls that read the plan run behind it on the
    same stream.  One whose only updates were captured holds its ids from the graph's first replay on: calls
    outside of the graph wait for that."""

    def __init__(self, rows, adapters, device):
        need = L.lora_multi_plan_bytes(rows, adapters)
        if not need:
            raise ValueError(f"a plan has 0 to 2^24 rows and 1 to 65535 adapters, got {rows} and {adapters}")
        self.rows, self.adapters = rows, adapters
        self.buffer = torch.empty(need, dtype=torch.uint8, device=device)
        self.filled = False               # calls refuse a plan before its first update

    def update(self, ids):
        """ids [rows], a contiguous int32 or int64 CUDA tensor: the adapter of each row, anything outside
        0 .. adapters - 1 for none."""
        _check_ids(ids)
        if ids.shape[0] != self.rows or ids.device != self.buffer.device:
            raise ValueError(f"ids must be [{self.rows}] on {self.buffer.device}, got {tuple(ids.shape)} on {ids.device}")
        L.need_current("ids", ids.device)
        L.lora_multi_plan(self.rows, self.adapters, ids, self.buffer)
        self.filled = True
        return self


def _check_ids(ids):
    if ids.dim() != 1 or ids.dtype not in (torch.int32, torch.int64) or not ids.is_contiguous():
        raise ValueError(f"ids must be a contiguous one-dimensional int32 or int64 tensor, got {tuple(ids.shape)} "
                         f"{ids.dtype} with strides {ids.stride()}")


def adapter_plan(ids, adapters):
    """The plan of a batch whose row i has adapter ids[i] of `adapters`, or none where the id is outside
    0 .. adapters - 1.  Made on the device, on the current stream; nothing waits for it.  One plan serves
    all projections of the batch, forward and backward."""
    _check_ids(ids)
    if not ids.is_cuda:
        raise ValueError(f"ids must be a CUDA tensor, got one on {ids.device}")
    L.need_current("ids", ids.device)
    return AdapterPlan(ids.shape[0], adapters, ids.device).update(ids)
