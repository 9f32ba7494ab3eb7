"""The ring's protocol with the numbers of slots and query buffers that it has beside sums in shared memory (up to 32 rows of a key head)."""
import pytest

import test_tree_protocol_host as model

# slots of a K and of a V tile, of the ring, queries' buffers, row tiles, warpgroups: d = 64, 128 (up to 16 rows; more), 256, 512
CONFIGS = [(1, 1, 12, 2, 1, 2), (1, 1, 6, 2, 1, 2), (1, 1, 5, 2, 1, 2), (2, 2, 6, 2, 1, 1), (2, 2, 5, 2, 1, 1), (4, 2, 5, 1, 1, 1), (4, 2, 5, 2, 1, 1), (4, 2, 6, 2, 1, 1)]
ROOM = {64: 229376, 128: 229376, 256: 231424, 512: 231424}  # bytes of shared memory for queries, ring and sums


@pytest.mark.parametrize("nc,nv,nslot,nqb,rt,wg", CONFIGS)
@pytest.mark.parametrize("seed", range(100, 106))
def test_ring_protocol_beside_sums(nc, nv, nslot, nqb, rt, wg, seed):
    model.test_ring_protocol(nc, nv, nslot, nqb, rt, wg, seed)


@pytest.mark.parametrize("d", [64, 128, 256, 512])
def test_rooms(d):
    """Every number of rows up to 32 gets one of those configurations, and all of it fits."""
    slot, most, wg, dv = (16384, 12, 2, 64) if d == 64 else (32768, 6, 2 if d == 128 else 1, min(d, 256))
    for rows in range(1, 33):
        q_rows = -(-rows // 8) * 8
        q, sums = q_rows * 2 * d, wg * dv * 4 * q_rows
        room = ROOM[d] - sums
        buffers = 2 if (room - 2 * q) // slot >= (10 if d == 64 else 5) else 1
        slots = min(most, (room - buffers * q) // slot)
        per = max(1, d // 128)
        assert (per, max(1, dv // 128), slots, buffers, 1, wg) in CONFIGS
        assert buffers * q + slots * slot + sums <= ROOM[d]
