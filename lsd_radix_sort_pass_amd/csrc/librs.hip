// librs.hip -- the sorts, and the mixture-of-experts calls around them, which use
// the sorts' launch and argument helpers.
#include "rs.hip"

#include "experts.hip"
