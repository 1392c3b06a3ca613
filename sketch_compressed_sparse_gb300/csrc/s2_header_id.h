// Which s2.h a binary was compiled from: the build defines S2_HEADER_ID, a word
// made of the header's contents.
#pragma once

#define S2_WORD_(w) #w
#define S2_WORD(w) S2_WORD_(w)
#ifdef S2_HEADER_ID
#define S2_HEADER_WORD S2_WORD(S2_HEADER_ID)
#else
#define S2_HEADER_WORD "unknown"
#endif
