// Which way os_attention_decode_shared reads its prefixes. Host code, from what the host knows: the
// sizes of the tables.
#pragma once

#include <cstdint>

namespace oss {

// Prefixes that cost little to read again are read by every sequence: the paged decode's
// kernel, over two sequences for each of the batch, and the join, two launches for three. The
// rule goes by the bytes that are read again if every prefix fills its row of the table, and no
// group is empty.
// From a graph, read again / on the tensor cores (sequences, heads, prefix): 4, 32 / 8, 1000 (12 MB):
// 10.5 / 15.6 us; 16, 8 / 1, 4000 (31): 13.1 / 16.8; 4, 32 / 8, 4000 (49): 14.8 / 17.2; 16, 32 / 8, 1000
// (61): 15.3 / 16.8; 37 in 5 groups, 16 / 2 of 64, 5001 (82): 19.9 / 16.6; 4, 32 / 8, 8000 (98): 20.9 / 20.8;
// 32, 32 / 8, 1000 (127): 22.2 / 17.4. Launched one by one, 24 us of the host against 30:
// on the GPU the two meet at 65 MB or so, with the host at twice that.
constexpr int64_t kReadAgain = int64_t(80) << 20;
// Groups may be empty, and the host does not know which: in the worst case all sequences are in one, and
// all but one of them read again. That bound is a looser one, since with a sequence in every
// group nothing is read twice and the decode's kernel is the better one at any length. From a graph,
// decode's kernel / tensor cores, 32 / 8 heads, as many groups as sequences; all sequences in one group: 16, 2000
// tokens (at most 123 MB): 20.7 / 15.9 us; 16, 4000 (246): 31.0 / 17.1; 64, 1000 (258): 38.6 / 26.2; 16, 16000
// (983): 91.2 / 27.5; 64, 16000 (4129): 335 / 43.6. One in each: 16, 2000: 30.5 / 42.4; 16, 4000: 49.9 /
// 60.9; 64, 1000: 54.8 / 73.1; 16, 16000: 162 / 170; 64, 16000: 617 / 618. At 256 MB either way
// loses 11 to 18 us where it is the wrong one; above, the loss of the first grows.
constexpr int64_t kReadAgainMost = int64_t(256) << 20;
constexpr int kPairGroups = 64;  // (every sequence looks its group up)

// blocks: of up to 16 query heads of a key head, each of which reads the keys and values; tokens: that a
// row of the prefix table has room for; token_bytes: of its keys and values. With blocks
// (from a graph, again / tensor cores): 1 sequence, 128 / 1 heads, 16000 tokens (57 MB): 19.2 / 16.8; 4, 128 / 1,
// 8000 (127): 23.6 / 16.6; 16, 64 / 1, 4000 (129): 24.5 / 16.4; 1, 128 / 1, 65536 (235): 37.0 / 28.6; 4, 128 / 1,
// 40000 (635): 71.6 / 29.9.
inline bool read_by_every_sequence(int64_t batch, int64_t groups, int64_t blocks, int64_t tokens, int64_t token_bytes) {
  const int64_t again = batch * blocks > groups ? batch * blocks - groups : 0, most = batch * blocks - 1;
  return groups <= kPairGroups && again * tokens <= kReadAgain / token_bytes && most * tokens <= kReadAgainMost / token_bytes;
}

}  // namespace oss
