"""fp64 CPU oracle of the operators around attention (test infrastructure only):
page bookkeeping of a serving step, and the per-head RMS norm with the rotary
position rotation, its backward pass included."""
from __future__ import annotations

import numpy as np

PAGE = 16


def extend_pages(block_table, seq_lens, new_lens, free_pages, free_count, max_tokens, num_pages):
    """Sequence by sequence: a page is taken from the end of the free list whenever a
    token begins one.  Sequences with impossible lengths stay as they are; from the first
    one whose pages or tokens do not fit on, all do.  Returns a dict of the outputs and
    the set of faults found ("index", "pages")."""
    table = np.array(block_table, dtype=np.int64)
    free = [int(x) for x in free_pages]
    faults = set()
    count = int(free_count)
    if count < 0 or count > num_pages:
        faults.add("index")
        count = 0
    lens, cu, pos, slots = [], [0], [], []
    full = False
    for b, (have, add) in enumerate(zip((int(x) for x in seq_lens), (int(x) for x in new_lens))):
        if have < 0 or add < 0 or have + add > table.shape[1] * PAGE:
            faults.add("index")
            add = 0
        need = -(-(have + add) // PAGE) - -(-have // PAGE) if add else 0
        if full or len(pos) + add > max_tokens or need > count:
            full = True
            faults.add("pages")
            add = 0
        for t in range(have, have + add):
            if t % PAGE == 0:
                count -= 1
                table[b, t // PAGE] = free[count]
            page = int(table[b, t // PAGE])
            if not 0 <= page < num_pages:
                faults.add("index")
            pos.append(t)
            slots.append(page * PAGE + t % PAGE if 0 <= page < num_pages else -1)
        lens.append(have + add)
        cu.append(len(pos))
    pad = max_tokens - len(pos)
    return dict(table=table, lens=np.array(lens, np.int64), cu=np.array(cu, np.int64),
                positions=np.array(pos + [0] * pad, np.int64),
                slots=np.array(slots + [-1] * pad, np.int64), left=count), faults


def rotation(table, positions, pair_axis, D, interleaved):
    """[T, D, D] rotation matrices: y = R x turns pair j of the first rot elements."""
    table = np.asarray(table, np.float64)
    positions = np.asarray(positions)
    rot = table.shape[1]
    T = positions.shape[1]
    R = np.tile(np.eye(D), (T, 1, 1))
    for j in range(rot // 2):
        u, v = (2 * j, 2 * j + 1) if interleaved else (j, j + rot // 2)
        axis = 0 if pair_axis is None else int(pair_axis[j])
        rows = table[positions[axis]]
        c, s = rows[:, j], rows[:, rot // 2 + j]
        R[:, u, u], R[:, u, v], R[:, v, u], R[:, v, v] = c, -s, s, c
    return R


def norm_rope(x, weight, R, eps):
    """y = R (w * x / sqrt(mean(x^2) + eps)) for x [T, H, D]; weight None: y = R x."""
    x = np.asarray(x, np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    return np.einsum("tij,thj->thi", R, x)


def norm_rope_backward(x, weight, R, dy, eps):
    """(dx, dw) of norm_rope for the gradient dy [T, H, D] (dw None without a weight)."""
    x = np.asarray(x, np.float64)
    g = np.einsum("tij,thi->thj", R, np.asarray(dy, np.float64))
    if weight is None:
        return g, None
    rstd = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xhat = x * rstd
    wg = g * np.asarray(weight, np.float64)
    return rstd * (wg - xhat * (wg * xhat).mean(-1, keepdims=True)), (g * xhat).sum((0, 1))
