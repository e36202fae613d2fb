"""CPU oracle of a verification step's two edges: block reservation, Q / K / V
staging and logit rules, in plain Python and numpy fp64, one row after the
other.  TEST INFRASTRUCTURE ONLY, like the rest of this package.
"""

from __future__ import annotations

import numpy as np

PAGE = 16
BAD_BLOCK, BAD_PARENT, BAD_WINDOW, BAD_LENGTH = 1, 2, 8, 128
POOL_EMPTY, BAD_SLOT, BAD_PARAM, EMPTY_MASK = 256, 512, 1024, 2048


def _depths(parent):
    """Depth of every node, or None if the parents are not topological."""
    depth = []
    for j, p in enumerate(parent):
        if (j == 0 and p != -1) or (j > 0 and not 0 <= p < j):
            return None
        depth.append(0 if j == 0 else depth[p] + 1)
    return depth


def reserve(cu, parent, ctx, tables, free_list, free_count, num_blocks, max_rows, total_rows,
            pos_offset=None):
    """(err, state) of sv_reserve_kv; the arrays given are not changed."""
    tables = np.array(tables, dtype=np.int32)
    R, width = tables.shape
    slots = np.full(total_rows, -1, np.int32)
    positions = np.full(total_rows, -1, np.int32)
    taken = np.full(R, -1, np.int32)
    err, asked, left = 0, 0, int(free_count)
    for i in range(R):
        c0, c1, n = int(cu[i]), int(cu[i + 1]), int(cu[i + 1]) - int(cu[i])
        if n < 1 or n > max_rows or c0 < 0 or c1 > total_rows:
            err |= BAD_WINDOW
            continue
        if ctx[i] < 0 or ctx[i] + n > width * PAGE:
            err |= BAD_LENGTH
            continue
        depth = list(range(n)) if parent is None else _depths([int(p) for p in parent[c0:c1]])
        t0, t1 = int(ctx[i]) // PAGE, -(-(int(ctx[i]) + n) // PAGE)
        part = tables[i, t0:t1]
        new = [t for t in range(t0, t1) if tables[i, t] == -1]
        bad = bool((part < -1).any() or (part >= num_blocks).any())
        bad |= bool(ctx[i] % PAGE and part[0] == -1)
        bad |= bool(new) and new != list(range(t1 - len(new), t1))
        err |= BAD_BLOCK if bad else 0
        err |= BAD_PARENT if depth is None else 0
        if bad or depth is None:
            continue
        asked += len(new)
        if new and asked > free_count:
            err |= POOL_EMPTY
            continue
        taken[i] = len(new)
        for t in new:
            left -= 1
            if 0 <= free_list[left] < num_blocks:
                tables[i, t] = free_list[left]
            else:
                err |= BAD_BLOCK
        for j in range(n):
            block = tables[i, (ctx[i] + j) // PAGE]
            if block >= 0:
                slots[c0 + j] = block * PAGE + (ctx[i] + j) % PAGE
                positions[c0 + j] = ctx[i] + depth[j] + (0 if pos_offset is None else pos_offset[i])
    return err, {"tables": tables, "count": left, "slots": slots, "positions": positions,
                 "taken": taken}


def stage(x, weight, eps, positions, inv_freq, rotary_dim, freq_axis=None, interleaved=False,
          scale=1.0):
    """(value, magnitude) fp64 [rows][heads][dim] of normed and rotated heads x;
    the magnitude is what the two terms of each element add up to in absolute
    value.  positions: [axes][rows]."""
    x = np.asarray(x, np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    y, mag = x.copy(), np.abs(x)
    for j in range(rotary_dim // 2):
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + rotary_dim // 2)
        axis = 0 if freq_axis is None else int(freq_axis[j])
        t = positions[axis].astype(np.float64) * float(inv_freq[j])
        c, s = scale * np.cos(t)[:, None], scale * np.sin(t)[:, None]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
        mag[..., a] = mag[..., b] = abs(scale) * (np.abs(x[..., a]) + np.abs(x[..., b]))
    return y, mag


def shape_logits(cu, parent, tokens, logits, history=None, history_len=None, prompt_len=None,
                 repetition=None, frequency=None, presence=None, bias_begin=None, bias_token=None,
                 bias_value=None, mask=None, mask_row=None):
    """(value, magnitude) fp64 [rows][vocab] of well-formed requests; the
    magnitude is the sum of the absolute values of what is added up."""
    y = np.array(logits, np.float64)
    V = y.shape[1]
    mag = np.abs(y)
    pen = repetition is not None or frequency is not None or presence is not None
    for i in range(len(cu) - 1):
        c0, c1 = int(cu[i]), int(cu[i + 1])
        for r in range(c0, c1):
            if pen:
                rho = 1.0 if repetition is None else float(repetition[i])
                f = 0.0 if frequency is None else float(frequency[i])
                p = 0.0 if presence is None else float(presence[i])
                n = 0 if history is None else int(history_len[i])
                k = 0 if history is None or prompt_len is None else int(prompt_len[i])
                said, seen = {}, set()
                for t in range(n):
                    v = int(history[i][t])
                    seen.add(v)
                    if t >= k:
                        said[v] = said.get(v, 0) + 1
                node = r - c0
                while node > 0:
                    v = int(tokens[c0 + node])
                    seen.add(v)
                    said[v] = said.get(v, 0) + 1
                    node = int(parent[c0 + node])
                for v in seen:
                    if not 0 <= v < V:
                        continue
                    x, c = y[r, v], said.get(v, 0)
                    x = x / rho if x > 0 else x * rho
                    y[r, v] = x - (f * c + p * (c > 0))
                    mag[r, v] = abs(x) + abs(f) * c + abs(p) * (c > 0)
            if bias_begin is not None:
                done = set()
                for t in range(int(bias_begin[i]), int(bias_begin[i + 1])):
                    v = int(bias_token[t])
                    if 0 <= v < V and v not in done:
                        done.add(v)
                        y[r, v] += float(bias_value[t])
                        mag[r, v] += abs(float(bias_value[t]))
            m = -1 if mask is None else r if mask_row is None else int(mask_row[r])
            if m >= 0:
                bits = (np.asarray(mask[m]).astype(np.uint32)[:, None] >> np.arange(32, dtype=np.uint32)) & 1
                let = bits.reshape(-1)[:V].astype(bool)
                if let.any():
                    y[r, ~let] = -np.inf
    return y, mag
